"""The gated linear recurrence on the GPU against float64 on the CPU, within bounds
that run along with the recurrence (seqops_ref.scan_errors, scan_back_errors)."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seqops_ref as ref  # noqa: E402
from seqops_ref import DT, d, near  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


CASES = [
    # B, L, C, x, gate, h, state, layout
    (1, 1, 1, "f32", "f32", "f32", True, "dense"),
    (2, 2, 5, "bf16", "f32", "bf16", True, "dense"),
    (1, 4, 8, "bf16", "bf16", "f32", False, "dense"),
    (3, 17, 9, "f32", "f32", "bf16", True, "padded"),
    (1, 65, 127, "bf16", "f32", "f32", True, "padded"),
    (2, 128, 128, "bf16", "bf16", "bf16", True, "fused"),
    (1, 129, 130, "f32", "f32", "f32", False, "time"),
    (2, 515, 70, "bf16", "bf16", "f32", True, "time"),
    (3, 1111, 101, "bf16", "f32", "f32", True, "fused"),
    (1, 2600, 264, "bf16", "bf16", "bf16", True, "dense"),
    (1, 9000, 24, "f32", "f32", "f32", True, "dense"),
    (150, 3, 40, "bf16", "bf16", "bf16", True, "dense"),
    (1, 300, 4100, "bf16", "bf16", "f32", True, "dense"),
]
MODES = [("log", "plain"), ("log", "blend"), ("log", "unit"), ("logit", "plain"), ("logit", "blend"), ("logit", "unit")]


def place(x, layout):
    B, L, C = x.shape
    if layout == "padded":
        buf = torch.full((B, L + 2, C + 5), float("nan"), dtype=x.dtype, device="cuda")
        buf[:, 1:-1, 3:C + 3] = x.cuda()
        return buf[:, 1:-1, 3:C + 3]
    if layout == "fused":
        buf = torch.full((B, L, 2 * C), float("nan"), dtype=x.dtype, device="cuda")
        buf[..., C:] = x.cuda()
        return buf[..., C:]
    if layout == "time":
        return x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    return x.cuda()


def make(case, decay, seed):
    """Gates from strong decays to memories of thousands of tokens, and resets."""
    B, L, C, xt, gt, ht, state, layout = case
    announce("gated scan", case, decay, seed)
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((B, L, C), generator=gen).to(DT[xt])
    strength = torch.exp(torch.empty((B, 1, C)).uniform_(-9.0, 3.0, generator=gen))
    if decay == "log":
        g = -strength * torch.rand((B, L, C), generator=gen)
        g = torch.where(torch.rand((B, L, C), generator=gen) < 0.002, torch.full_like(g, -float("inf")), g)
    else:
        g = -strength.log() + torch.randn((B, L, C), generator=gen)
    g = g.to(DT[gt])
    h0 = torch.randn((B, C), generator=gen).cuda() if state else None
    return place(x, layout), place(g, layout), h0, gen


@pytest.mark.parametrize("decay,inputs", MODES)
@pytest.mark.parametrize("case", CASES)
def test_forward(case, decay, inputs):
    import delta_rule_linear_amd as drl
    x, g, h0, _ = make(case, decay, case[1])
    m = dict(decay=decay, inputs=inputs)
    h, last = drl.dr_gated_scan_fwd(x, g, h0, out_dtype=DT[case[5]], **m)
    want, wlast = ref.scan_forward(d(x), d(g), d(h0), decay, inputs)
    e, elast = ref.scan_errors(d(x), d(g), d(h0), decay, inputs)
    near(h, want, e, "h")
    near(last, wlast, elast, "h_final")


@pytest.mark.parametrize("decay,inputs", MODES)
@pytest.mark.parametrize("case", CASES)
def test_backward(case, decay, inputs):
    import delta_rule_linear_amd as drl
    B, L, C, xt, gt, ht, state, layout = case
    x, g, h0, gen = make(case, decay, L + 1)
    m = dict(decay=decay, inputs=inputs)
    h, _ = drl.dr_gated_scan_fwd(x, g, h0, out_dtype=DT[ht], **m)
    h = place(h.cpu(), layout)
    dh = place(torch.randn((B, L, C), generator=gen).to(DT[xt if L % 2 else ht]), layout)
    dlast = torch.randn((B, C), generator=gen).cuda() if state else None
    for to in ("f32", "bf16") if L < 200 else (ht,):
        got = drl.dr_gated_scan_bwd(x, g, h0, h, dh, dlast, grad_dtype=DT[to], **m)
        want = ref.scan_backward(d(x), d(g), d(h0), d(h), d(dh), d(dlast), decay, inputs)
        ex, eg, e0 = ref.scan_back_errors(d(x), d(g), want, d(dh), d(dlast), decay, inputs)
        near(got["dx"], want["dx"], ex, "dx")
        near(got["dgate"], want["dgate"], eg, "dgate")
        near(got["dh0"], want["dh0"], e0, "dh0")


@pytest.mark.parametrize("decay,inputs", MODES)
@pytest.mark.parametrize("B,C,xt,gt,ht", [(1, 1, "f32", "f32", "f32"), (3, 7, "bf16", "f32", "bf16"),
                                          (256, 2048, "bf16", "bf16", "bf16"), (33, 1001, "f32", "f32", "bf16"),
                                          (2, 9, "bf16", "bf16", "f32")])
def test_step_is_the_forward_of_one_token(B, C, xt, gt, ht, decay, inputs):
    import delta_rule_linear_amd as drl
    x, g, h0, _ = make((B, 3, C, xt, gt, ht, True, "dense"), decay, C)
    m = dict(decay=decay, inputs=inputs, out_dtype=DT[ht])
    state, last = h0.clone(), h0.clone()
    for t in range(3):
        h = drl.dr_gated_scan_step(state, x[:, t].contiguous(), g[:, t].contiguous(), **m)
        want, last = drl.dr_gated_scan_fwd(x[:, t:t + 1], g[:, t:t + 1], last, **m)
        assert torch.equal(h, want[:, 0]) and torch.equal(state, last)


def test_sequences_in_parts_and_states_in_place():
    """The tokens in two calls, the state carried in place, within the bounds."""
    import delta_rule_linear_amd as drl
    x, g, h0, _ = make((2, 700, 75, "f32", "f32", "f32", True, "dense"), "logit", 3)
    m = dict(decay="logit", inputs="unit")
    want, wlast = ref.scan_forward(d(x), d(g), d(h0), "logit", "unit")
    e, elast = ref.scan_errors(d(x), d(g), d(h0), "logit", "unit")
    for k in (0, 1, 333, 700):
        s = h0.clone()
        h1, got = drl.dr_gated_scan_fwd(x[:, :k], g[:, :k], s, h_final=s, **m)
        assert got is s
        h2, _ = drl.dr_gated_scan_fwd(x[:, k:], g[:, k:], s, h_final=s, **m)
        near(torch.cat([h1, h2], 1), want, e, "h")
        near(s, wlast, elast, "h_final")
    e = x[:, :0]
    got = drl.dr_gated_scan_bwd(e, e, h0, e, e, h0, **m)
    assert torch.equal(got["dh0"], h0) and got["dx"].shape == e.shape


def test_resets_long_memories_and_bad_values():
    import delta_rule_linear_amd as drl
    inf = float("inf")
    gen = torch.Generator().manual_seed(7)
    # a constant decay of 1 - 2^-14 over 40000 tokens: a rounded to 24 bits would be off by 2^-11 of 1 - a
    g = torch.full((1, 40000, 8), -2.0 ** -14, device="cuda")
    x = torch.ones((1, 40000, 8), device="cuda")
    for inputs in ("plain", "blend", "unit"):
        h, last = drl.dr_gated_scan_fwd(x, g, None, decay="log", inputs=inputs)
        a = torch.tensor(-2.0 ** -14, dtype=torch.float64).exp()
        c = {"plain": torch.ones(()).double(), "blend": 1 - a, "unit": (1 - a * a).sqrt()}[inputs]
        want = (c * (1 - a ** 40000) / (1 - a)).expand(1, 8)
        # each token rounds the state once or twice, at random
        assert ((d(last) - want).abs() <= 1e-5 * want).all(), inputs
    # no decay at all
    h, last = drl.dr_gated_scan_fwd(torch.ones((1, 5000, 8), device="cuda"), torch.zeros((1, 5000, 8), device="cuda"),
                                    decay="log")
    assert torch.equal(h[0, :, 0].cpu(), torch.arange(1.0, 5001.0)) and (last == 5000).all()
    # a reset forgets exactly, whatever the state was
    x, g = torch.randn((1, 600, 11), generator=gen).cuda(), -torch.rand((1, 600, 11), generator=gen).cuda()
    g[0, 300] = -inf
    for inputs in ("plain", "blend", "unit"):
        m = dict(decay="log", inputs=inputs)
        h, _ = drl.dr_gated_scan_fwd(x, g, torch.full((1, 11), 1e30, device="cuda"), **m)
        assert torch.equal(h[:, 300], x[:, 300])
        got = drl.dr_gated_scan_bwd(x, g, None, h, torch.ones_like(h), **m)
        assert (got["dgate"][0, 300] == 0).all()
    # NaN: the later tokens of its channel, and no others
    clean, _ = drl.dr_gated_scan_fwd(x, g, None, decay="log")
    x[0, 200, 4] = float("nan")
    h, _ = drl.dr_gated_scan_fwd(x, g, None, decay="log")
    bad = torch.zeros(h.shape, dtype=torch.bool)
    bad[0, 200:, 4] = True
    assert torch.equal(h.cpu()[~bad], clean.cpu()[~bad]) and torch.isnan(h.cpu()[bad]).all()
    # saturated logits
    g = torch.tensor([200.0, -200.0, inf, -inf], device="cuda").reshape(1, 4, 1).repeat(1, 1, 16)
    x = torch.ones((1, 4, 16), device="cuda")
    h, _ = drl.dr_gated_scan_fwd(x, g, None, decay="logit", inputs="blend")
    assert torch.equal(h[0, :, 0].cpu(), torch.tensor([0.0, 1.0, 1.0, 1.0]))
    got = drl.dr_gated_scan_bwd(x, g, None, h, torch.ones_like(h), decay="logit", inputs="unit")
    assert all(torch.isfinite(t).all() for t in got.values())


def test_outputs_streams_and_replay():
    import delta_rule_linear_amd as drl
    x, g, h0, gen = make((2, 1500, 204, "bf16", "bf16", "bf16", True, "dense"), "logit", 9)
    dh = torch.randn(x.shape, generator=gen).to(torch.bfloat16).cuda()
    m = dict(decay="logit", inputs="unit")

    def chain(stream=None):
        h, last = drl.dr_gated_scan_fwd(x, g, h0, stream=stream, **m)
        got = drl.dr_gated_scan_bwd(x, g, h0, h, dh, stream=stream, **m)
        return (h, last) + tuple(got.values())

    base = chain()
    buf = torch.full((2, 1502, 210), 5.0, device="cuda")
    out = buf[:, 1:-1, 3:207]
    h, none = drl.dr_gated_scan_fwd(x, g, h0, h=out, want_state=False, **m)
    assert h is out and none is None and torch.equal(out, base[0])
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


@pytest.mark.parametrize("decay,inputs", MODES)
def test_gradients_against_differences(decay, inputs):
    """Central differences, h = 2^-12: a gate's third derivative along a direction
    grows with its weight in the state, below 2000 times the loss's magnitude: off by
    less than 2^-13 of it."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(6)
    x, dh = torch.randn((2, 19, 12), generator=gen).cuda(), torch.randn((2, 19, 12), generator=gen).cuda()
    g = (-0.2 - torch.rand((2, 19, 12), generator=gen)).cuda() * (1 if decay == "log" else -1)
    h0, dlast = torch.randn((2, 12), generator=gen).cuda(), torch.randn((2, 12), generator=gen).cuda()
    h, _ = drl.dr_gated_scan_fwd(x, g, h0, decay=decay, inputs=inputs)
    got = drl.dr_gated_scan_bwd(x, g, h0, h, dh, dlast, decay=decay, inputs=inputs)
    base = {"x": d(x), "g": d(g), "h0": d(h0)}

    def loss(v):
        y, last = ref.scan_forward(v["x"], v["g"], v["h0"], decay, inputs)
        return float((d(dh) * y).sum() + (d(dlast) * last).sum())

    s = 2.0 ** -12
    for n, gn in (("x", "dx"), ("g", "dgate"), ("h0", "dh0")):
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (loss({**base, n: base[n] + s * v}) - loss({**base, n: base[n] - s * v})) / (2 * s)
        assert abs(float((d(got[gn]) * v).sum()) - want) <= 2.0 ** -13 * float((d(got[gn]).abs() * v.abs()).sum()), n


def test_refusals_of_the_binding():
    import delta_rule_linear_amd as drl
    x = torch.randn(2, 5, 16, device="cuda")
    with pytest.raises(ValueError, match="decay"):
        drl.dr_gated_scan_fwd(x, x, decay="token")
    with pytest.raises(ValueError, match="inputs"):
        drl.dr_gated_scan_fwd(x, x, decay="log", inputs="half")
    with pytest.raises(ValueError, match="gate has shape"):
        drl.dr_gated_scan_fwd(x, x[:, :3], decay="log")
    with pytest.raises(drl.DeltaRuleError, match="gate must have"):
        drl.dr_gated_scan_fwd(x, x.to(torch.bfloat16), decay="log")
    with pytest.raises(ValueError, match="h0 has shape"):
        drl.dr_gated_scan_fwd(x, x, x[:, 0, :8].contiguous(), decay="log")
    with pytest.raises(drl.DeltaRuleError, match="overlaps"):
        drl.dr_gated_scan_fwd(x, x, h=x, decay="log")
    with pytest.raises(ValueError, match="must be a"):
        drl.dr_gated_scan_fwd(x[0], x[0], decay="log")
    with pytest.raises(ValueError, match="contiguous"):
        drl.dr_gated_scan_step(torch.zeros(2, 16, device="cuda"), x[:, 0], x[:, 1].contiguous(), decay="log")
    with pytest.raises(TypeError):
        drl.dr_gated_scan_bwd(x, x, None, x, x, decay="log", grad_dtype=torch.float16)
