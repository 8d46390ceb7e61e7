"""Layer norm on the GPU against float64 on the CPU.

Bounds.  With u = 2^-24: the mean of D values is off by at most D u mean|x|; the
variance comes from x - mean, so it and rstd are off by (D + 4) u relative, plus
what the mean's error moves them by.  y is a product of those with three more
roundings: |y - want| <= (2 D + 16) u (|n| + |m| rstd + 1) |w| + 4 u |b| where
m is the mean of |x|.  Sums over rows of R terms are off by R u of the sum of
absolute values.  bf16 results add half a step, 2^-8."""
import pytest

import linattn_ref as ref
from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def near(got, want, bound, what, bf16=False):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if bf16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    err = (got - want).abs()
    assert (err <= bound + 1e-37).all(), f"{what}: worst {float((err / (bound + 1e-37)).max()):.3g} of the bound"


def data(shape, per_head, dtype, dy_dtype, layout, seed, shift=0.5, scale=1.0):
    announce("layer norm", shape, per_head, dtype, dy_dtype, layout, seed)
    B, H, L, D = shape
    gen = torch.Generator().manual_seed(seed)
    t = {"x": (shift + scale * torch.randn(shape, generator=gen)).to(DT[dtype]),
         "dy": torch.randn(shape, generator=gen).to(DT[dy_dtype])}
    for n in t:
        if layout == "token":
            t[n] = t[n].transpose(1, 2).contiguous().cuda().transpose(1, 2)
        elif layout == "padded":   # rows of a buffer whose other values are NaN
            pad = 8 if D % 8 == 0 else 3
            buf = torch.full((B, H, L + 1, D + pad), float("nan"), dtype=t[n].dtype, device="cuda")
            buf[:, :, :L, :D] = t[n].cuda()
            t[n] = buf[:, :, :L, :D]
        else:
            t[n] = t[n].cuda()
    w = (H, D) if per_head else (D,)
    t["w"] = (1 + 0.3 * torch.randn(w, generator=gen)).cuda()
    t["b"] = (0.3 * torch.randn(w, generator=gen)).cuda()
    return t


def wide(w, per_head):
    w = w.double().cpu()
    return w[None, :, None] if per_head else w


def check_fwd(t, per_head, eps, got, out, w=True, b=True):
    x = t["x"].double().cpu()
    y, mean, rstd = ref.norm_forward(x, t["w"].double().cpu() if w else None, t["b"].double().cpu() if b else None, eps)
    D = x.shape[-1]
    m = x.abs().mean(-1)
    near(got[1], mean, (D + 2) * U * m, "mean")
    # the variance: relative (D + 4) u, and the mean's error squared
    dmean = (D + 2) * U * m
    rel = (D + 6) * U + (dmean * rstd) ** 2 + 4 * U * m * rstd
    near(got[2], rstd, rstd * rel, "rstd")
    n = ((x - mean[..., None]) * rstd[..., None]).abs()
    wa = wide(t["w"], per_head).abs() if w else torch.ones(())
    ba = wide(t["b"], per_head).abs() if b else torch.zeros(())
    bound = wa * (n * (rel + 6 * U)[..., None] + ((dmean + 2 * U * m) * rstd)[..., None]) + 4 * U * (ba + n * wa)
    near(got[0], y, bound, "y", out == "bf16")


CASES = [
    # B, H, L, D, per_head, dtype, out, layout
    (1, 1, 1, 1, False, "f32", "f32", "dense"),
    (2, 3, 5, 8, True, "bf16", "bf16", "dense"),
    (2, 3, 70, 64, True, "bf16", "f32", "token"),
    (1, 5, 33, 63, True, "bf16", "bf16", "padded"),
    (3, 4, 100, 128, True, "bf16", "bf16", "token"),
    (2, 2, 65, 128, False, "f32", "bf16", "padded"),
    (1, 2, 40, 200, True, "f32", "f32", "dense"),
    (1, 1, 300, 1001, False, "f32", "f32", "padded"),
    (1, 1, 9, 512, False, "bf16", "bf16", "dense"),
    (2, 1, 31, 1024, False, "bf16", "bf16", "token"),
    (1, 1, 1100, 2048, False, "bf16", "bf16", "dense"),
    (1, 1, 7, 2049, False, "f32", "f32", "dense"),
    (1, 2, 5, 4096, True, "bf16", "f32", "token"),
    (1, 1, 17, 8184, False, "f32", "bf16", "padded"),
    (1, 1, 3, 16384, False, "bf16", "bf16", "dense"),
    (1, 1, 2, 16383, False, "f32", "f32", "dense"),
    (2, 16, 1500, 48, True, "bf16", "bf16", "dense"),
    # even widths that are no multiples of 8
    (1, 1, 1, 2, False, "bf16", "bf16", "dense"),
    (2, 3, 37, 100, True, "bf16", "bf16", "token"),
    (1, 2, 65, 250, True, "f32", "f32", "padded"),
    (1, 1, 19, 1002, False, "bf16", "f32", "dense"),
    (1, 1, 5, 6002, False, "f32", "bf16", "dense"),
    (1, 1, 3, 16382, False, "bf16", "bf16", "dense"),
]


@pytest.mark.parametrize("B,H,L,D,per_head,dtype,out,layout", CASES)
def test_forward(B, H, L, D, per_head, dtype, out, layout):
    import delta_rule_linear_amd as drl
    t = data((B, H, L, D), per_head, dtype, dtype, layout, D)
    got = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"], eps=1e-5, out_dtype=DT[out])
    check_fwd(t, per_head, 1e-5, got, out)


@pytest.mark.parametrize("B,H,L,D,per_head,dtype,out,layout", CASES)
def test_backward(B, H, L, D, per_head, dtype, out, layout):
    import delta_rule_linear_amd as drl
    other = {"bf16": "f32", "f32": "bf16"}
    t = data((B, H, L, D), per_head, dtype, dtype if D % 2 else other[dtype], layout, D + 1)
    _, mean, rstd = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"])
    g = drl.dr_layernorm_bwd(t["x"], t["w"], mean, rstd, t["dy"], grad_dtype=DT[out])
    d = lambda v: v.double().cpu()  # noqa: E731
    dx, dw, db = ref.norm_backward(d(t["x"]), d(t["w"]), d(mean), d(rstd), d(t["dy"]), per_head)
    # n = (x - mean) rstd is off by 3 u |n| (the subtraction is rounded once)
    n = ((d(t["x"]) - d(mean)[..., None]) * d(rstd)[..., None]).abs()
    dy = d(t["dy"]).abs()
    tt = dy * wide(t["w"], per_head).abs()
    r = d(rstd)[..., None]
    bound = r * U * (8 * tt + (D + 8) * tt.mean(-1, keepdim=True) + (D + 12) * n * (tt * n).mean(-1, keepdim=True))
    near(g["dx"], dx, bound, "dx", out == "bf16")
    over = (0, 2) if per_head else (0, 1, 2)
    terms = B * L if per_head else B * H * L
    near(g["dweight"], dw, (terms + 8) * U * (dy * n).sum(over), "dweight")
    near(g["dbias"], db, (terms + 8) * U * dy.sum(over), "dbias")


def test_shapes_and_absent_weights():
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((6, 4, 64), generator=gen).cuda()
    w, b = torch.randn((4, 64), generator=gen).cuda(), torch.randn((4, 64), generator=gen).cuda()
    # [N, H, D] with a weight per head is [N, H, 1, D]; [B, L, D] with one weight [B, 1, L, D]
    y, mean, rstd = drl.dr_layernorm_fwd(x, w, b)
    assert y.shape == x.shape and mean.shape == (6, 4)
    y4, _, _ = drl.dr_layernorm_fwd(x[:, :, None], w, b)
    assert torch.equal(y, y4[:, :, 0])
    y3, _, _ = drl.dr_layernorm_fwd(x, w[0], b[0])
    y2, m2, r2 = drl.dr_layernorm_fwd(x.reshape(24, 64), w[0], b[0])
    assert torch.equal(y3.reshape(24, 64), y2)
    plain, _, _ = drl.dr_layernorm_fwd(x)
    ones, _, _ = drl.dr_layernorm_fwd(x, torch.ones(64, device="cuda"), torch.zeros(64, device="cuda"))
    assert torch.equal(plain, ones)
    g = drl.dr_layernorm_bwd(x, None, mean, rstd, y, per_head=True)
    assert g["dweight"].shape == (4, 64)
    g1 = drl.dr_layernorm_bwd(x, torch.ones(4, 64, device="cuda"), mean, rstd, y)
    assert all(torch.equal(g[n], g1[n]) for n in g)
    g0 = drl.dr_layernorm_bwd(x, None, mean, rstd, y, per_head=True, want_sums=False)
    assert g0["dweight"] is None and torch.equal(g0["dx"], g["dx"])
    # no rows
    e = x[:0]
    y, mean, rstd = drl.dr_layernorm_fwd(e, w, b)
    assert y.shape == (0, 4, 64)
    g = drl.dr_layernorm_bwd(e, w, mean, rstd, y)
    assert not g["dweight"].any() and not g["dbias"].any()


def test_constant_large_and_bad_rows():
    """A row of one value has variance 0 (rstd = 1 / sqrt(eps)); a large mean
    costs no accuracy of the variance beyond the inputs' own; a NaN stays in its
    row (and in the sums over rows)."""
    import delta_rule_linear_amd as drl
    x = torch.full((3, 128), 7.0, device="cuda")
    y, mean, rstd = drl.dr_layernorm_fwd(x, eps=1e-4)
    assert not y.any() and (mean == 7).all() and torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)
    t = data((1, 1, 50, 128), False, "f32", "f32", "dense", 2, shift=1000.0)
    check_fwd(t, False, 1e-5, drl.dr_layernorm_fwd(t["x"], t["w"], t["b"]), "f32")
    x = torch.randn((5, 128)).cuda()
    ref_y, _, _ = drl.dr_layernorm_fwd(x)
    x[2, 7] = float("nan")
    y, _, _ = drl.dr_layernorm_fwd(x)
    assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3, 4]], ref_y[[0, 1, 3, 4]])


def test_output_layout_and_streams_and_replay():
    import delta_rule_linear_amd as drl
    t = data((2, 4, 300, 128), True, "bf16", "bf16", "dense", 5)
    y0, mean, rstd = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"])
    g0 = drl.dr_layernorm_bwd(t["x"], t["w"], mean, rstd, t["dy"])
    buf = torch.full((2, 300, 4, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    y = buf[..., :128].transpose(1, 2)
    got, _, _ = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"], y=y)
    assert got is y and torch.equal(y, y0) and (buf[..., 128:] == 5).all()
    torch.cuda.synchronize()
    many = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        many.append(drl.dr_layernorm_bwd(t["x"], t["w"], mean, rstd, t["dy"], stream=s))
    torch.cuda.synchronize()
    for g in many:
        assert all(torch.equal(g[n], g0[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1, m1, r1 = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"])
        g1 = drl.dr_layernorm_bwd(t["x"], t["w"], m1, r1, t["dy"])
    for n in range(4):
        t["x"].copy_(torch.randn(t["x"].shape, generator=torch.Generator().manual_seed(n)))
        graph.replay()
        torch.cuda.synchronize()
        e, em, er = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"])
        ge = drl.dr_layernorm_bwd(t["x"], t["w"], em, er, t["dy"])
        assert torch.equal(y1, e) and all(torch.equal(g1[k], ge[k]) for k in ge)


def test_gradients_against_differences():
    """Central differences of the float64 forward with h = 2^-10: its third
    derivatives along a direction are below 100 times the loss's magnitude, so
    the differences are off by less than 2^-13 of it."""
    import delta_rule_linear_amd as drl
    t = data((2, 3, 20, 40), True, "f32", "f32", "dense", 8)
    _, mean, rstd = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"])
    g = drl.dr_layernorm_bwd(t["x"], t["w"], mean, rstd, t["dy"])
    gen = torch.Generator().manual_seed(2)
    base = {n: t[n].double().cpu() for n in ("x", "w", "b")}
    dy = t["dy"].double().cpu()
    loss = lambda v: float((dy * ref.norm_forward(v["x"], v["w"], v["b"], 1e-5)[0]).sum())  # noqa: E731
    h = 2.0 ** -10
    for n, gn in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        d = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (loss({**base, n: base[n] + h * d}) - loss({**base, n: base[n] - h * d})) / (2 * h)
        got = float((g[gn].double().cpu() * d).sum())
        size = float((g[gn].double().cpu().abs() * d.abs()).sum())
        assert abs(got - want) <= 2.0 ** -13 * size, (n, got, want)


def test_attention_and_norm_trained_together():
    """Attention, per-head norm, loss and back, as a layer runs them, against
    the same chain in float64: bf16 activations between the steps, so each
    entry may be off by the roundings of o, y and dO (2^-8 each) carried
    through, i.e. by 2^-5 of a gradient's 2-norm."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(11)
    B, H, Hk, L, D = 2, 4, 2, 300, 64
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v = (r(B, L, n, D).to(torch.bfloat16).cuda().transpose(1, 2) for n in (Hk, Hk, H))
    la = -0.1 * torch.rand((H,), generator=gen).cuda()
    w, b = (1 + 0.1 * r(H, D)).cuda(), (0.1 * r(H, D)).cuda()
    dy = r(B, L, H, D).to(torch.bfloat16).cuda().transpose(1, 2)
    o, S = drl.dr_linear_attn_fwd(q, k, v, la, decay="head", out_dtype=torch.bfloat16)
    y, mean, rstd = drl.dr_layernorm_fwd(o, w, b)
    gn = drl.dr_layernorm_bwd(o, w, mean, rstd, dy)
    g = drl.dr_linear_attn_bwd(q, k, v, la, None, gn["dx"], decay="head", grad_dtype=torch.bfloat16)
    d = lambda t: t.double().cpu()  # noqa: E731
    a = ref.gates(la, "head", B, H, L)
    Q, K, V = ref.heads(d(q), H), ref.heads(d(k), H), d(v)
    wo, wS = ref.forward(Q, K, V, a)
    wy, wm, wr = ref.norm_forward(wo, d(w), d(b), 1e-5)
    wdx, wdw, wdb = ref.norm_backward(wo, d(w), wm, wr, d(dy), True)
    dq, dk, dv, dla, _ = ref.backward(Q, K, V, a, None, wdx, None)
    for got, want, what in ((y, wy, "y"), (S, wS, "S"), (gn["dweight"], wdw, "dweight"), (gn["dbias"], wdb, "dbias"),
                            (g["dq"], ref.shared(dq, Hk), "dq"), (g["dk"], ref.shared(dk, Hk), "dk"), (g["dv"], dv, "dv"),
                            (g["dlog_alpha"], dla.sum((0, 2)), "dlog_alpha")):
        err = float((d(got) - want).norm() / want.norm())
        assert err <= 2.0 ** -5, (what, err)
    # serving: the next tokens from the prefill's state, each normed
    for n in range(3):
        q1, k1, v1 = (r(B, m, D).to(torch.bfloat16).cuda() for m in (Hk, Hk, H))
        o1 = drl.dr_linear_attn_step(S, q1, k1, v1, la, decay="head")
        y1, _, _ = drl.dr_layernorm_fwd(o1, w, b, out_dtype=torch.bfloat16)
        wo1, wS = ref.forward(ref.heads(d(q1)[:, :, None], H), ref.heads(d(k1)[:, :, None], H), d(v1)[:, :, None],
                              ref.gates(la, "head", B, H, 1), wS)
        wy1, _, _ = ref.norm_forward(wo1, d(w), d(b), 1e-5)
        assert float((d(y1) - wy1[:, :, 0]).norm() / wy1.norm()) <= 2.0 ** -5


def test_refusals_of_the_binding():
    import delta_rule_linear_amd as drl
    x = torch.randn(4, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="same shape"):
        drl.dr_layernorm_fwd(x, w, torch.ones(3, 64, device="cuda"))
    with pytest.raises(ValueError, match="weight has shape"):
        drl.dr_layernorm_fwd(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError, match="weight must be"):
        drl.dr_layernorm_fwd(x, w.to(torch.bfloat16))
    with pytest.raises(ValueError, match="channels of a row"):
        drl.dr_layernorm_fwd(x.transpose(1, 2))
    with pytest.raises(TypeError):
        drl.dr_layernorm_fwd(x.half())
    with pytest.raises(drl.DeltaRuleError, match="eps"):
        drl.dr_layernorm_fwd(x, eps=-1.0)
    with pytest.raises(drl.DeltaRuleError, match="overlaps"):
        drl.dr_layernorm_fwd(x, w, y=x)
    with pytest.raises(drl.DeltaRuleError, match="D=16385"):
        drl.dr_layernorm_fwd(torch.zeros(2, 16385, device="cuda"))
    _, mean, rstd = drl.dr_layernorm_fwd(x, w)
    with pytest.raises(drl.DeltaRuleError, match="workspace"):
        drl.dr_layernorm_bwd(x, w, mean, rstd, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="dy has shape"):
        drl.dr_layernorm_bwd(x, w, mean, rstd, x[:2])
