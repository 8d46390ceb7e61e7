"""The short causal convolution on the GPU against float64 on the CPU, within bounds
from the sums of absolute values (seqops_ref.conv_bounds)."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seqops_ref as ref  # noqa: E402
from seqops_ref import DT, U, d, near  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


CASES = [
    # B, L, C, W, dtype, out, silu, state, layout
    (1, 1, 1, 2, "f32", "f32", True, True, "dense"),
    (2, 3, 5, 4, "bf16", "bf16", True, True, "dense"),
    (1, 2, 8, 8, "f32", "f32", True, True, "dense"),        # fewer tokens than taps
    (3, 7, 9, 8, "bf16", "f32", False, True, "padded"),
    (2, 5, 16, 3, "bf16", "bf16", False, False, "dense"),
    (1, 65, 127, 4, "bf16", "bf16", True, True, "padded"),
    (1, 64, 128, 5, "f32", "bf16", True, False, "fused"),
    (2, 300, 136, 4, "bf16", "bf16", True, True, "time"),
    (3, 1111, 100, 4, "bf16", "f32", True, True, "fused"),
    (1, 2050, 258, 6, "f32", "f32", True, True, "dense"),
    (2, 515, 70, 7, "bf16", "bf16", True, False, "padded"),
    (1, 9000, 24, 2, "bf16", "bf16", True, True, "dense"),
    (70, 1, 40, 4, "bf16", "bf16", True, True, "dense"),
    (1, 700, 4100, 4, "bf16", "bf16", True, True, "dense"),
]


def rows(B, L, C, dtype, layout, gen):
    x = torch.randn((B, L, C), generator=gen).to(DT[dtype])
    if layout == "padded":      # starts anywhere, among NaN
        buf = torch.full((B, L + 2, C + 5), float("nan"), dtype=x.dtype, device="cuda")
        buf[:, 1:-1, 3:C + 3] = x.cuda()
        return buf[:, 1:-1, 3:C + 3]
    if layout == "fused":       # a part of a projection's rows
        buf = torch.full((B, L, 3 * C), float("nan"), dtype=x.dtype, device="cuda")
        buf[..., C:2 * C] = x.cuda()
        return buf[..., C:2 * C]
    if layout == "time":        # tokens in front of batches
        return x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    return x.cuda()


def make(case, seed):
    B, L, C, W, dtype, out, silu, state, layout = case
    announce("short convolution", case, seed)
    gen = torch.Generator().manual_seed(seed)
    x = rows(B, L, C, dtype, layout, gen)
    w, b = torch.randn((C, W), generator=gen).cuda(), (0.5 * torch.randn(C, generator=gen)).cuda()
    st = torch.randn((B, W - 1, C), generator=gen).to(DT[dtype]).cuda() if state else None
    return x, w, (b if C % 3 else None), st, "silu" if silu else "none", gen


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    import delta_rule_linear_amd as drl
    x, w, b, st, act, _ = make(case, case[2])
    y, last = drl.dr_short_conv_fwd(x, w, b, st, activation=act, out_dtype=DT[case[5]])
    args = d(x), d(w), d(b), d(st), act == "silu"
    want = ref.conv_forward(*args)
    near(y, want[0], ref.conv_bounds(*args, want)[1], "y")
    assert torch.equal(d(last), want[1])
    if st is not None:
        # in place, and the tokens in two calls
        s2 = st.clone()
        k = case[1] // 2
        y1, got = drl.dr_short_conv_fwd(x[:, :k], w, b, s2, activation=act, out_dtype=DT[case[5]], state_out=s2)
        assert got is s2
        y2, _ = drl.dr_short_conv_fwd(x[:, k:], w, b, s2, activation=act, out_dtype=DT[case[5]], state_out=s2)
        assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(s2, last)


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    import delta_rule_linear_amd as drl
    B, L, C, W, dtype, out, silu, state, layout = case
    x, w, b, st, act, gen = make(case, case[2] + 1)
    dy = rows(B, L, C, dtype if C % 2 else "f32", layout, gen)
    dlast = torch.randn((B, W - 1, C), generator=gen).cuda() if state else None
    g = drl.dr_short_conv_bwd(x, w, b, st, dy, dlast, activation=act, grad_dtype=DT[out])
    args = d(x), d(w), d(b), d(st)
    want = ref.conv_backward(*args, d(dy), d(dlast), silu)
    # dz: the slope moves by at most half of z's error, and is off by a few u of its terms
    z, s = want["z"], torch.sigmoid(want["z"])
    dz_err = torch.zeros_like(z)
    if silu:
        ez, _ = ref.conv_bounds(*args, True, ref.conv_forward(*args, True))
        dz_err = d(dy).abs() * (0.5 * ez + (12 + 4 * z.abs()) * U * s * (1 + z.abs() * (1 - s)))
    mag, dz = torch.zeros_like(want["past"]), want["dz"].abs()
    for j in range(W):
        mag[:, j:j + L] += d(w)[:, j].abs() * (dz_err + (W + 3) * U * dz)
    if dlast is not None:
        mag[:, L:] += 2 * U * d(dlast).abs()
    mag = mag + U * torch.cat([want["dstate"], want["dx"]], 1).abs()
    near(g["dx"], want["dx"], mag[:, W - 1:], "dx")
    near(g["dstate"], want["dstate"], mag[:, :W - 1], "dstate")
    n = B * L + 8
    bw = torch.stack([((dz_err + n * U * dz) * want["past"][:, j:j + L].abs()).sum((0, 1)) for j in range(W)], -1)
    near(g["dweight"], want["dweight"], bw, "dweight")
    near(g["dbias"], want["dbias"], (dz_err + n * U * dz).sum((0, 1)), "dbias")


@pytest.mark.parametrize("B,C,W,dtype,out", [(1, 1, 4, "f32", "f32"), (3, 7, 2, "bf16", "bf16"), (5, 8, 8, "bf16", "f32"),
                                             (256, 2048, 4, "bf16", "bf16"), (33, 1001, 4, "f32", "bf16"),
                                             (2, 65, 3, "bf16", "bf16")])
def test_step_is_the_forward_of_one_token(B, C, W, dtype, out):
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(C)
    w, b = torch.randn((C, W), generator=gen).cuda(), torch.randn(C, generator=gen).cuda()
    st = torch.randn((B, W - 1, C), generator=gen).to(DT[dtype]).cuda()
    one, all_ = st.clone(), st.clone()
    for n in range(W + 1):
        x = torch.randn((B, C), generator=gen).to(DT[dtype]).cuda()
        y = drl.dr_short_conv_step(one, x, w, b, out_dtype=DT[out])
        want, all_ = drl.dr_short_conv_fwd(x[:, None], w, b, all_, out_dtype=DT[out])
        assert torch.equal(y, want[:, 0]) and torch.equal(one, all_)


def test_bad_values_stay_in_their_window():
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((1, 200, 19), generator=gen).cuda()
    w = torch.randn((19, 4), generator=gen).cuda()
    clean, _ = drl.dr_short_conv_fwd(x, w)
    x[0, 63, 5] = float("nan")
    x[0, 100, 18] = -float("inf")
    y, _ = drl.dr_short_conv_fwd(x, w)
    bad = torch.zeros(y.shape, dtype=torch.bool)
    bad[0, 63:67, 5] = True
    bad[0, 100:104, 18] = True
    assert torch.equal(y.cpu()[~bad], clean.cpu()[~bad])
    assert torch.isnan(y[0, 63:67, 5]).all()
    # SiLU of -inf is 0, of +inf infinite
    want = torch.where(w[18].flip(0) > 0, 0.0, float("inf"))
    assert torch.equal(y[0, 100:104, 18], want)
    empty, st = drl.dr_short_conv_fwd(x[:, :0], w, None, x[:, :3].contiguous())
    assert empty.shape == (1, 0, 19) and torch.equal(st, x[:, :3])
    g = drl.dr_short_conv_bwd(x[:, :0], w, None, None, x[:, :0], x[:, 3:6].contiguous())
    assert torch.equal(g["dstate"], x[:, 3:6]) and not g["dweight"].any() and not g["dbias"].any()


def test_outputs_streams_and_replay():
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(5)
    x, dy = (torch.randn((2, 500, 204), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    w, b = torch.randn((204, 4), generator=gen).cuda(), torch.randn(204, generator=gen).cuda()
    st = torch.randn((2, 3, 204), generator=gen).to(torch.bfloat16).cuda()

    def chain(stream=None):
        y, last = drl.dr_short_conv_fwd(x, w, b, st, stream=stream)
        g = drl.dr_short_conv_bwd(x, w, b, st, dy, stream=stream)
        return (y, last) + tuple(g.values())

    base = chain()
    buf = torch.full((2, 502, 210), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 1:-1, 3:207]
    y, none = drl.dr_short_conv_fwd(x, w, b, st, y=out, want_state=False)
    assert y is out and none is None and torch.equal(out, base[0])
    out.fill_(5.0)
    assert (buf == 5.0).all()
    torch.cuda.synchronize()
    many = [chain(s) for s in [torch.cuda.Stream() for _ in range(3)]]
    torch.cuda.synchronize()
    for got in many:
        assert all(torch.equal(p, q) for p, q in zip(base, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain()
    for n in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(n)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, chain()))


def test_gradients_against_differences():
    """Central differences, h = 2^-10; third derivatives along a direction are below
    100 times the loss's magnitude: off by less than 2^-13 of it."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(6)
    x, dy = torch.randn((2, 21, 12), generator=gen).cuda(), torch.randn((2, 21, 12), generator=gen).cuda()
    w, b = (0.5 * torch.randn((12, 4), generator=gen)).cuda(), torch.randn(12, generator=gen).cuda()
    st, dlast = torch.randn((2, 3, 12), generator=gen).cuda(), torch.randn((2, 3, 12), generator=gen).cuda()
    g = drl.dr_short_conv_bwd(x, w, b, st, dy, dlast)
    base = {"x": d(x), "w": d(w), "b": d(b), "st": d(st)}

    def loss(v):
        y, last, _ = ref.conv_forward(v["x"], v["w"], v["b"], v["st"], True)
        return float((d(dy) * y).sum() + (d(dlast) * last).sum())

    h = 2.0 ** -10
    for n, gn in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("st", "dstate")):
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (loss({**base, n: base[n] + h * v}) - loss({**base, n: base[n] - h * v})) / (2 * h)
        assert abs(float((d(g[gn]) * v).sum()) - want) <= 2.0 ** -13 * float((d(g[gn]).abs() * v.abs()).sum()), n


def test_refusals_of_the_binding():
    import delta_rule_linear_amd as drl
    x = torch.randn(2, 5, 16, device="cuda")
    w = torch.ones((16, 4), device="cuda")
    with pytest.raises(ValueError, match="activation"):
        drl.dr_short_conv_fwd(x, w, activation="relu")
    with pytest.raises(ValueError, match="weight has shape"):
        drl.dr_short_conv_fwd(x, w[:8])
    with pytest.raises(drl.DeltaRuleError, match="W=9"):
        drl.dr_short_conv_fwd(x, torch.ones((16, 9), device="cuda"))
    with pytest.raises(drl.DeltaRuleError, match="W=1"):
        drl.dr_short_conv_fwd(x, torch.ones((16, 1), device="cuda"))
    with pytest.raises(ValueError, match="state has shape"):
        drl.dr_short_conv_fwd(x, w, None, x[:, :2].contiguous())
    with pytest.raises(TypeError, match="state must be"):
        drl.dr_short_conv_fwd(x, w, None, x[:, :3].to(torch.bfloat16))
    with pytest.raises(ValueError, match="channels of a row"):
        drl.dr_short_conv_fwd(x.transpose(1, 2), torch.ones((5, 4), device="cuda"))
    with pytest.raises(drl.DeltaRuleError, match="overlaps"):
        drl.dr_short_conv_fwd(x, w, y=x)
    with pytest.raises(ValueError, match="contiguous"):
        drl.dr_short_conv_step(torch.zeros(2, 3, 16, device="cuda"), x[:, 0], w)
    with pytest.raises(drl.DeltaRuleError, match="workspace"):
        drl.dr_short_conv_bwd(x, w, None, None, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
