"""RMS norm on the GPU against float64 on the CPU.

Bounds, u = 2^-24.  The sum s = x + r is rounded once.  The mean of D squares is off
by (D + 4) u of itself, rstd by half of that and 4 u; y has three more roundings:
|y| (D + 12) u.  Sums over R rows are off by R u of the sum of absolute values.
bf16 results add half a step, 2^-8; e4m3 codes half of theirs."""
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


def rows(shape, dtype, layout, gen, scale=1.0):
    B, H, L, D = shape
    x = (scale * torch.randn(shape, generator=gen)).to(DT[dtype])
    if layout == "token":
        return x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    if layout == "padded":   # rows of a buffer whose other values are NaN, starting anywhere
        buf = torch.full((B, H, L + 1, D + 3), float("nan"), dtype=x.dtype, device="cuda")
        buf[:, :, 1:, 1:D + 1] = x.cuda()
        return buf[:, :, 1:, 1:D + 1]
    return x.cuda()


CASES = [
    # B, H, L, D, per_head, dtype, residual, out, layout
    (1, 1, 1, 1, False, "f32", None, "f32", "dense"),
    (1, 2, 3, 5, True, "bf16", "f32", "bf16", "dense"),
    (2, 3, 5, 8, True, "bf16", "bf16", "bf16", "dense"),
    (2, 3, 70, 64, True, "bf16", "f32", "f32", "token"),
    (1, 5, 33, 63, True, "bf16", None, "bf16", "padded"),
    (3, 4, 100, 128, True, "bf16", "bf16", "bf16", "token"),
    (2, 2, 65, 129, False, "f32", "f32", "bf16", "padded"),
    (1, 2, 40, 200, True, "f32", None, "f32", "dense"),
    (1, 1, 300, 1001, False, "f32", "f32", "f32", "padded"),
    (1, 1, 9, 512, False, "bf16", "bf16", "bf16", "dense"),
    (2, 1, 31, 1024, False, "bf16", "f32", "bf16", "token"),
    (1, 1, 1100, 2048, False, "bf16", "bf16", "bf16", "dense"),
    (1, 1, 7, 2049, False, "f32", "f32", "f32", "dense"),
    (1, 2, 5, 4096, True, "bf16", "f32", "f32", "token"),
    (1, 1, 17, 8184, False, "f32", None, "bf16", "padded"),
    (1, 1, 3, 16384, False, "bf16", "f32", "bf16", "dense"),
    (1, 1, 2, 16383, False, "f32", "f32", "f32", "dense"),
    (2, 16, 1500, 48, True, "bf16", None, "bf16", "dense"),
]


def make(case, seed):
    B, H, L, D, per_head, dtype, res, out, layout = case
    announce("RMS norm", case, seed)
    gen = torch.Generator().manual_seed(seed)
    x = rows((B, H, L, D), dtype, layout, gen)
    r = None if res is None else rows((B, H, L, D), res, layout, gen, 3.0)
    w = (1 + 0.3 * torch.randn((H, D) if per_head else (D,), generator=gen)).cuda()
    return x, r, w, (d(w)[None, :, None] if per_head else d(w)), gen


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    import delta_rule_linear_amd as drl
    x, r, w, wide, _ = make(case, case[3])
    D = case[3]
    y, rstd, total = drl.dr_rmsnorm_fwd(x, w, r, eps=1e-5, out_dtype=DT[case[7]])
    s, wy, wr = ref.rms_forward(d(x), d(r), wide, 1e-5)
    near(rstd, wr, (D + 8) * U * wr, "rstd")
    near(y, wy, (D + 12) * U * wy.abs(), "y")
    if r is None:
        assert total is None
    else:
        assert total.dtype == r.dtype
        near(total, s, U * s.abs(), "total")


@pytest.mark.parametrize("block", (128, 0))
@pytest.mark.parametrize("case", CASES)
def test_eight_bits(case, block):
    import delta_rule_linear_amd as drl
    x, r, w, wide, _ = make(case, case[3] + 7)
    D = case[3]
    y, scale, rstd, total = drl.dr_rmsnorm_fwd_e4m3(x, w, r, eps=1e-5, block=block)
    assert y.dtype == torch.float8_e4m3fn
    s, wy, wr = ref.rms_forward(d(x), d(r), wide, 1e-5)
    near(rstd, wr, (D + 8) * U * wr, "rstd")
    if r is not None:
        near(total, s, U * s.abs(), "total")
    n = block or D
    parts = torch.nn.functional.pad(wy, (0, -D % n)).unflatten(-1, (-1, n))
    want = (parts.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    near(scale, want, (D + 16) * U * want, "scale")
    # the codes: half a step of the quotient, which is off by the roundings of y and scale
    v = wy / want.repeat_interleave(n, -1)[..., :D]
    got = d(y.float())
    off = 2 * (D + 16) * U * v.abs()
    bound = ref.e4m3_step(torch.maximum(v.abs() + off, got.abs())) / 2 + off
    assert ((got - v).abs() <= bound).all(), float(((got - v).abs() / bound).max())
    assert float(got.abs().max()) <= 448


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    import delta_rule_linear_amd as drl
    B, H, L, D, per_head, dtype, res, out, layout = case
    x, _, w, wide, gen = make(case, D + 1)
    other = {"bf16": "f32", "f32": "bf16"}
    dy = rows((B, H, L, D), dtype if D % 2 else other[dtype], layout, gen)
    ds = None if res is None else rows((B, H, L, D), res, layout, gen)
    _, rstd, _ = drl.dr_rmsnorm_fwd(x, w)
    g = drl.dr_rmsnorm_bwd(x, w, rstd, dy, ds, grad_dtype=DT[out])
    r = d(rstd)[..., None]
    dx, terms = ref.rms_backward(d(x), wide, d(rstd), d(dy), d(ds))
    n, t = (d(x) * r).abs(), (d(dy) * wide).abs()
    bound = r * U * (8 * t + (D + 12) * n * (t * n).mean(-1, keepdim=True))
    if ds is not None:
        bound = bound + 2 * U * (dx.abs() + d(ds).abs())
    near(g["dx"], dx, bound, "dx")
    over = (0, 2) if per_head else (0, 1, 2)
    near(g["dweight"], terms.sum(over), ((B * L if per_head else B * H * L) + 8) * U * terms.abs().sum(over), "dweight")


def test_shapes_layouts_and_absent_weights():
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(1)
    x, r = torch.randn((6, 4, 64), generator=gen).cuda(), torch.randn((6, 4, 64), generator=gen).cuda()
    w = torch.randn((4, 64), generator=gen).cuda()
    y, rstd, total = drl.dr_rmsnorm_fwd(x, w, r)
    y4, _, _ = drl.dr_rmsnorm_fwd(x[:, :, None], w, r[:, :, None])
    assert torch.equal(y, y4[:, :, 0]) and torch.equal(total, x + r)
    y3, _, _ = drl.dr_rmsnorm_fwd(x, w[0], r)
    y2, _, _ = drl.dr_rmsnorm_fwd(x.reshape(24, 64), w[0], r.reshape(24, 64))
    assert torch.equal(y3.reshape(24, 64), y2)
    plain, _, _ = drl.dr_rmsnorm_fwd(x)
    ones, _, _ = drl.dr_rmsnorm_fwd(x, torch.ones(64, device="cuda"))
    assert torch.equal(plain, ones)
    # a residual shared by all rows, and an output inside a larger buffer, which keeps the rest
    shared = r[:1, :1].expand(6, 4, 64)
    buf = torch.full((6, 5, 70), 5.0, device="cuda")
    out = buf[:, :4, 3:67]
    y, rstd, total = drl.dr_rmsnorm_fwd(x, w, shared, y=out)
    want, _, _ = drl.dr_rmsnorm_fwd(x, w, shared.contiguous())
    assert y is out and torch.equal(out, want)
    out.fill_(5.0)
    assert (buf == 5.0).all()
    g = drl.dr_rmsnorm_bwd(x, None, rstd, y, per_head=True)
    g1 = drl.dr_rmsnorm_bwd(x, torch.ones(4, 64, device="cuda"), rstd, y)
    assert all(torch.equal(g[n], g1[n]) for n in g)
    g0 = drl.dr_rmsnorm_bwd(x, None, rstd, y, per_head=True, want_sums=False)
    assert g0["dweight"] is None and torch.equal(g0["dx"], g["dx"])
    e = x[:0]
    y, rstd, total = drl.dr_rmsnorm_fwd(e, w, r[:0])
    assert y.shape == total.shape == (0, 4, 64)
    y8, scale, _, _ = drl.dr_rmsnorm_fwd_e4m3(e, w)
    assert scale.shape == (0, 4, 1)
    assert not drl.dr_rmsnorm_bwd(e, w, rstd, y)["dweight"].any()


@pytest.mark.parametrize("rows,D,dtype", [(5, 64, "f32"), (700, 129, "bf16"), (3000, 2048, "bf16"), (40, 5001, "f32"), (9, 5, "f32")])
def test_the_sum_in_the_residuals_place(rows, D, dtype):
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(D)
    x, r = (torch.randn((rows, D), generator=gen).to(DT[dtype]).cuda() for _ in range(2))
    y, rstd, total = drl.dr_rmsnorm_fwd(x, None, r)
    y8, scale, _, _ = drl.dr_rmsnorm_fwd_e4m3(x, None, r)
    for f in (lambda t: drl.dr_rmsnorm_fwd(x, None, t, total=t)[0], lambda t: drl.dr_rmsnorm_fwd_e4m3(x, None, t, total=t)[0]):
        t = r.clone()
        got = f(t)
        assert torch.equal(t, total)
        assert torch.equal(got, y) if got.dtype == y.dtype else torch.equal(got.view(torch.uint8), y8.view(torch.uint8))


def test_zero_tiny_large_and_bad_rows():
    import delta_rule_linear_amd as drl
    x = torch.zeros((4, 256), device="cuda")
    x[1] = 1e-30
    x[2] = 1e15
    x[3, :128] = 1.0
    for block in (128, 0):
        y, scale, rstd, _ = drl.dr_rmsnorm_fwd_e4m3(x, eps=1e-5, block=block)
        assert torch.isfinite(scale).all() and (y.float()[0] == 0).all() and (scale[0] == 2.0 ** -126).all()
        got = y.float() * scale.repeat_interleave(256 // scale.shape[-1], -1)
        _, want, wr = ref.rms_forward(d(x), None, None, 1e-5)
        near(rstd, wr, 300 * U * wr, "rstd")
        assert ((d(got) - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -126).all()
    # a NaN stays in its row, an infinity too: rstd is 0 there and its own value NaN
    x = torch.randn((5, 300), generator=torch.Generator().manual_seed(3)).cuda()
    clean, cs, _, _ = drl.dr_rmsnorm_fwd_e4m3(x)
    yc, _, _ = drl.dr_rmsnorm_fwd(x)
    x[1, 290] = float("nan")
    x[3, 5] = float("inf")
    y8, scale, rstd, _ = drl.dr_rmsnorm_fwd_e4m3(x)
    y, _, _ = drl.dr_rmsnorm_fwd(x)
    good = [0, 2, 4]
    assert torch.equal(y[good], yc[good]) and torch.equal(y8.float()[good], clean.float()[good])
    assert torch.equal(scale[good], cs[good])
    assert torch.isnan(y[1]).all() and torch.isnan(y8.float()[1]).all()
    assert rstd[3] == 0 and torch.isnan(y[3, 5]) and (y[3, :5] == 0).all()
    # an infinity that the weight makes: its block's scale is infinite, its codes NaN
    w = torch.ones(300, device="cuda")
    w[7] = float("inf")
    y8, scale, _, _ = drl.dr_rmsnorm_fwd_e4m3(x[:1], w)
    assert scale[0, 0] == float("inf") and torch.isnan(y8.float()[0, :128]).all()
    assert torch.isfinite(scale[0, 1:]).all() and torch.equal(y8.float()[0, 128:], clean.float()[0, 128:])


def test_streams_and_replay():
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(5)
    x, r, dy = (torch.randn((2, 300, 520), generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    w = torch.randn(520, generator=gen).cuda()

    def chain(stream=None):
        y, rstd, total = drl.dr_rmsnorm_fwd(x, w, r, stream=stream)
        y8, scale, _, _ = drl.dr_rmsnorm_fwd_e4m3(x, w, r, stream=stream)
        g = drl.dr_rmsnorm_bwd(total, w, rstd, dy, r, stream=stream)
        return y, rstd, total, y8.view(torch.uint8), scale, g["dx"], g["dweight"]

    base = chain()
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
    """Central differences of the float64 forward, h = 2^-10: third derivatives along a
    direction are below 100 times the loss's magnitude, so the differences are off
    by less than 2^-13 of it."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(2)
    x, dy, ds = (torch.randn((7, 40), generator=gen).cuda() for _ in range(3))
    r = torch.randn((7, 40), generator=gen).cuda()
    w = (1 + 0.3 * torch.randn(40, generator=gen)).cuda()
    _, rstd, total = drl.dr_rmsnorm_fwd(x, w, r)
    g = drl.dr_rmsnorm_bwd(total, w, rstd, dy, ds)
    base = {"x": d(x), "r": d(r), "w": d(w)}

    def loss(v):
        s, y, _ = ref.rms_forward(v["x"], v["r"], v["w"], 1e-5)
        return float((d(dy) * y).sum() + (d(ds) * s).sum())

    h = 2.0 ** -10
    for n, gn in (("x", "dx"), ("r", "dx"), ("w", "dweight")):
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (loss({**base, n: base[n] + h * v}) - loss({**base, n: base[n] - h * v})) / (2 * h)
        assert abs(float((d(g[gn]) * v).sum()) - want) <= 2.0 ** -13 * float((d(g[gn]).abs() * v.abs()).sum()), n


def test_refusals_of_the_binding():
    import delta_rule_linear_amd as drl
    x = torch.randn(4, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="residual has shape"):
        drl.dr_rmsnorm_fwd(x, w, x[:2])
    with pytest.raises(drl.DeltaRuleError, match="residual must have"):
        drl.dr_rmsnorm_fwd(x, w, x.to(torch.bfloat16))
    with pytest.raises(ValueError, match="there is none"):
        drl.dr_rmsnorm_fwd(x, w, total=torch.empty_like(x))
    with pytest.raises(TypeError, match="weight must be"):
        drl.dr_rmsnorm_fwd(x, w.to(torch.bfloat16))
    with pytest.raises(ValueError, match="block"):
        drl.dr_rmsnorm_fwd_e4m3(x, w, block=64)
    with pytest.raises(ValueError, match="block"):
        drl.dr_rmsnorm_fwd_e4m3(x, w, block=None)
    with pytest.raises(TypeError, match="y must be"):
        drl.dr_rmsnorm_fwd_e4m3(x, w, y=torch.empty_like(x))
    with pytest.raises(TypeError):
        drl.dr_rmsnorm_fwd(x, w, out_dtype=torch.float8_e4m3fn)
    with pytest.raises(drl.DeltaRuleError, match="overlaps"):
        drl.dr_rmsnorm_fwd(x, w, x.clone(), total=x)
    with pytest.raises(drl.DeltaRuleError, match="overlaps"):
        drl.dr_rmsnorm_fwd(x, w, y=x)
    _, rstd, _ = drl.dr_rmsnorm_fwd(x, w)
    with pytest.raises(drl.DeltaRuleError, match="workspace"):
        drl.dr_rmsnorm_bwd(x, w, rstd, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="ds has shape"):
        drl.dr_rmsnorm_bwd(x, w, rstd, x, x[:2])
