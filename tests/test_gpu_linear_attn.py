"""Linear attention with a decay per head on the GPU against float64 on the CPU
(tests/linattn_ref.py states where the bounds come from)."""
import math

import pytest

import linattn_ref as ref
from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows(gen, shape, dtype, layout="dense", scale=1.0):
    """[B,H,L,D] of N(0, 1) on the GPU: dense, a view of [B,L,H,D], or a view of
    longer rows of a buffer whose other values are NaN."""
    B, H, L, D = shape
    x = (scale * torch.randn(shape, generator=gen)).to(DT[dtype])
    if layout == "token":
        return x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    if layout == "padded":
        buf = torch.full((B, H, L + 5, D + 16), float("nan"), dtype=DT[dtype], device="cuda")
        buf[:, :, 2:L + 2, 8:D + 8] = x.cuda()
        return buf[:, :, 2:L + 2, 8:D + 8]
    return x.cuda()


def decays(gen, decay, B, H, L, lo=-0.1, hi=-0.001):
    if decay == "none":
        return None
    shape = (H,) if decay == "head" else (B, H, L)
    return (lo + (hi - lo) * torch.rand(shape, generator=gen)).cuda()


def problem(B, H, Hk, L, Dk, Dv, decay, dtype, layout="dense", seed=0, state=True, lo=-0.1, hi=-0.001, grad=False):
    announce("linear attention", B, H, Hk, L, Dk, Dv, decay, dtype, layout, seed, lo)
    gen = torch.Generator().manual_seed(seed)
    p = dict(q=rows(gen, (B, Hk, L, Dk), dtype, layout, Dk ** -0.5), k=rows(gen, (B, Hk, L, Dk), dtype, layout),
             v=rows(gen, (B, H, L, Dv), dtype, layout), la=decays(gen, decay, B, H, L, lo, hi),
             S0=torch.randn((B, H, Dk, Dv), generator=gen).cuda() if state else None)
    if grad:
        p["dO"] = rows(gen, (B, H, L, Dv), dtype, layout)
        p["dS"] = torch.randn((B, H, Dk, Dv), generator=gen).cuda() if state else None
    return p


def run_fwd(p, decay, out="f32", **kw):
    import delta_rule_linear_amd as drl
    return drl.dr_linear_attn_fwd(p["q"], p["k"], p["v"], p["la"], p["S0"], decay=decay, out_dtype=DT[out], **kw)


def run_bwd(p, decay, out="f32", **kw):
    import delta_rule_linear_amd as drl
    return drl.dr_linear_attn_bwd(p["q"], p["k"], p["v"], p["la"], p["S0"], p["dO"], p["dS"], decay=decay,
                                  grad_dtype=DT[out], **kw)


def check_fwd(p, decay, out="f32", got=None):
    o, S = run_fwd(p, decay, out) if got is None else got
    want, size = ref.reference(p["q"], p["k"], p["v"], p["la"], p["S0"], decay)
    n = ref.slack(o.shape[2], p["q"].shape[-1], o.shape[-1])
    ref.check(o, want["o"], size["o"], n, "o", out == "bf16")
    ref.check(S, want["S"], size["S"], n, "S")


def check_bwd(p, decay, out="f32", got=None):
    g = run_bwd(p, decay, out) if got is None else got
    want, size = ref.reference(p["q"], p["k"], p["v"], p["la"], p["S0"], decay, p["dO"], p["dS"])
    n = ref.slack(p["q"].shape[2], p["q"].shape[-1], p["v"].shape[-1])
    for name in ("dq", "dk", "dv"):
        ref.check(g[name], want[name], size[name], n, name, out == "bf16")
    ref.check(g["dS0"], want["dS0"], size["dS0"], n, "dS0")
    if decay == "none":
        assert g["dlog_alpha"] is None
    else:
        ref.check(g["dlog_alpha"], want["dlog_alpha"], size["dlog_alpha"], n, "dlog_alpha")


CASES = [
    # B, H, Hk, L, Dk, Dv, decay, dtype, out, layout
    (1, 1, 1, 1, 64, 64, "token", "bf16", "f32", "dense"),
    (2, 3, 3, 1, 128, 128, "head", "f32", "f32", "dense"),
    (1, 2, 2, 63, 64, 64, "head", "bf16", "bf16", "dense"),
    (1, 2, 1, 64, 128, 128, "token", "bf16", "f32", "token"),
    (2, 2, 2, 65, 128, 64, "token", "bf16", "bf16", "padded"),
    (1, 2, 2, 65, 64, 128, "none", "f32", "f32", "token"),
    (1, 6, 2, 130, 64, 96, "head", "bf16", "f32", "token"),
    (2, 4, 1, 200, 8, 8, "token", "bf16", "f32", "dense"),
    (1, 3, 3, 200, 128, 8, "token", "f32", "bf16", "padded"),
    (1, 2, 2, 200, 16, 128, "none", "bf16", "bf16", "dense"),
    (1, 3, 1, 129, 48, 104, "token", "bf16", "f32", "padded"),
    (1, 2, 2, 129, 72, 40, "head", "f32", "f32", "padded"),
    (3, 5, 5, 192, 120, 24, "token", "bf16", "f32", "token"),
    (1, 1, 1, 1000, 64, 32, "token", "bf16", "f32", "dense"),
    (1, 2, 1, 1030, 128, 128, "head", "bf16", "bf16", "token"),
    (1, 1, 1, 1100, 128, 128, "token", "f32", "f32", "dense"),
    (1, 4, 2, 777, 64, 64, "token", "f32", "f32", "token"),
]


@pytest.mark.parametrize("B,H,Hk,L,Dk,Dv,decay,dtype,out,layout", CASES)
def test_forward(B, H, Hk, L, Dk, Dv, decay, dtype, out, layout):
    check_fwd(problem(B, H, Hk, L, Dk, Dv, decay, dtype, layout, seed=L), decay, out)


@pytest.mark.parametrize("B,H,Hk,L,Dk,Dv,decay,dtype,out,layout", CASES)
def test_backward(B, H, Hk, L, Dk, Dv, decay, dtype, out, layout):
    check_bwd(problem(B, H, Hk, L, Dk, Dv, decay, dtype, layout, seed=L + 1, grad=True), decay, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lo,hi", [(-3.0, -0.5), (-200.0, -1.0), (0.0, 0.0), (0.0, 0.02)])
def test_strong_absent_and_growing_decays(dtype, lo, hi):
    p = problem(1, 2, 2, 300, 64, 64, "token", dtype, lo=lo, hi=hi, grad=True)
    check_fwd(p, "token")
    check_bwd(p, "token")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_decay_of_zero_starts_anew(dtype):
    p = problem(1, 2, 1, 200, 64, 64, "token", dtype, grad=True)
    for t in (0, 64, 65, 131):
        p["la"][:, :, t] = -math.inf
    check_fwd(p, "token")
    check_bwd(p, "token")
    g = run_bwd(p, "token")
    # nothing passes a reset: neither a gradient of its own nor one of S0, and no S0
    assert not g["dlog_alpha"][:, :, [0, 64, 65, 131]].any()
    S0 = p["S0"]
    p["S0"] = torch.zeros_like(S0)
    o0, _ = run_fwd(p, "token")
    p["S0"] = S0
    o1, _ = run_fwd(p, "token")
    assert torch.equal(o0, o1)
    assert not g["dS0"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequences_in_segments(dtype):
    """One or two sequences are cut into segments that are joined."""
    import delta_rule_linear_amd as drl
    p = problem(1, 1, 1, 4113, 128, 64, "token", dtype, grad=True, lo=-0.02, hi=0.0)
    d = drl.linattn_desc(1, 1, 1, 4113, 128, 64, drl.DR_BF16, drl.DR_F32, "token")
    assert drl.dr_linear_attn_fwd_workspace_bytes(d) > 0
    check_fwd(p, "token")
    check_bwd(p, "token")
    p = problem(1, 2, 1, 2500, 64, 128, "head", dtype, grad=True, lo=-0.01, hi=-0.0001)
    check_fwd(p, "head", "bf16")
    check_bwd(p, "head")


@pytest.mark.parametrize("decay", ["none", "head", "token"])
def test_without_states(decay):
    p = problem(2, 2, 2, 100, 64, 64, decay, "bf16", state=False, grad=True)
    check_fwd(p, decay)
    check_bwd(p, decay)
    o, S = run_fwd(p, decay, want_state=False)
    assert S is None
    g = run_bwd(p, decay, want_dS0=False)
    assert g["dS0"] is None


def test_state_in_place_split_and_step():
    """Two calls, the second on the first's state in place, and one token at a
    time, against one call."""
    import delta_rule_linear_amd as drl
    p = problem(2, 4, 2, 150, 64, 96, "token", "bf16")
    check_fwd(p, "token")
    S = p["S0"].clone()
    cut = lambda t, a, b: t[:, :, a:b]  # noqa: E731
    parts = []
    for a, b in ((0, 70), (70, 147)):
        o, S2 = drl.dr_linear_attn_fwd(cut(p["q"], a, b), cut(p["k"], a, b), cut(p["v"], a, b),
                                       cut(p["la"], a, b).contiguous(), S, decay="token", S_final=S)
        assert S2 is S
        parts.append(o)
    for t in range(147, 150):
        at = lambda x: x[:, :, t].contiguous()  # noqa: E731,B023
        parts.append(drl.dr_linear_attn_step(S, at(p["q"]), at(p["k"]), at(p["v"]), at(p["la"]), decay="token")[:, :, None])
    check_fwd(p, "token", got=(torch.cat(parts, 2), S))


STEPS = [
    (1, 1, 1, 64, 64, "head", "bf16", "bf16"),
    (3, 6, 2, 128, 128, "token", "bf16", "f32"),
    (5, 4, 4, 128, 64, "none", "f32", "f32"),
    (2, 3, 1, 8, 104, "token", "f32", "bf16"),
    (7, 2, 2, 120, 24, "head", "bf16", "f32"),
    (300, 8, 4, 64, 128, "token", "bf16", "f32"),
]


@pytest.mark.parametrize("N,H,Hk,Dk,Dv,decay,dtype,out", STEPS)
def test_step(N, H, Hk, Dk, Dv, decay, dtype, out):
    import delta_rule_linear_amd as drl
    announce("step", N, H, Hk, Dk, Dv, decay, dtype, out)
    gen = torch.Generator().manual_seed(N)
    q, k = (torch.randn((N, Hk, Dk), generator=gen).to(DT[dtype]).cuda() for _ in range(2))
    v = torch.randn((N, H, Dv), generator=gen).to(DT[dtype]).cuda()
    S = torch.randn((N, H, Dk, Dv), generator=gen).cuda()
    la = decays(gen, decay, N, H, 1)
    la = la[..., 0].contiguous() if decay == "token" else la
    want, size = ref.reference(q[:, :, None], k[:, :, None], v[:, :, None],
                               la[..., None] if decay == "token" else la, S, decay)
    o = drl.dr_linear_attn_step(S, q, k, v, la, decay=decay, out_dtype=DT[out])
    n = ref.slack(1, Dk, Dv)
    ref.check(o, want["o"][:, :, 0], size["o"][:, :, 0], n, "o", out == "bf16", two_terms=False)
    ref.check(S, want["S"], size["S"], n, "S")


def test_step_with_a_decay_of_zero_and_no_states():
    import delta_rule_linear_amd as drl
    S = torch.randn(2, 3, 64, 64).cuda()
    q, k, v = (torch.randn(2, 3, 64).cuda() for _ in range(3))
    la = torch.zeros(2, 3).cuda()
    la[0, 1] = -math.inf
    drl.dr_linear_attn_step(S, q, k, v, la, decay="token")
    assert torch.equal(S[0, 1], k[0, 1][:, None] * v[0, 1][None])
    e = torch.empty(0, 3, 64, device="cuda")
    o = drl.dr_linear_attn_step(S[:0], e, e, e, la[:0], decay="token")
    assert o.shape == (0, 3, 64)


def test_empty_calls():
    import delta_rule_linear_amd as drl
    p = problem(2, 2, 2, 0, 64, 64, "head", "bf16", grad=True)
    o, S = run_fwd(p, "head")
    assert o.shape == (2, 2, 0, 64) and torch.equal(S, p["S0"])
    g = run_bwd(p, "head")
    assert torch.equal(g["dS0"], p["dS"]) and not g["dlog_alpha"].any()
    p["S0"] = p["dS"] = None
    _, S = run_fwd(p, "head")
    assert not S.any()
    assert not run_bwd(p, "head")["dS0"].any()
    z = torch.empty(0, 2, 5, 64, device="cuda")
    o, S = drl.dr_linear_attn_fwd(z, z, z, decay="none")
    assert o.shape == (0, 2, 5, 64) and S.shape == (0, 2, 64, 64)
    g = drl.dr_linear_attn_bwd(z, z, z, torch.zeros(2, device="cuda"), None, z, decay="head")
    assert not g["dlog_alpha"].any()


def test_broadcast_rows_and_slices_of_one_projection():
    """q and k as slices of one [B, L, heads, 2 D] projection; v one row for
    every head (stride 0), whose gradient comes per head."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(3)
    B, H, L, D = 2, 4, 100, 64
    qk = torch.randn((B, L, H, 2 * D), generator=gen).to(torch.bfloat16).cuda()
    p = dict(q=qk[..., :D].transpose(1, 2), k=qk[..., D:].transpose(1, 2),
             v=torch.randn((B, 1, L, D), generator=gen).to(torch.bfloat16).cuda().expand(B, H, L, D),
             la=decays(gen, "head", B, H, L), S0=None, dS=None,
             dO=torch.randn((1, 1, 1, D), generator=gen).to(torch.bfloat16).cuda().expand(B, H, L, D))
    check_fwd(p, "head")
    check_bwd(p, "head")
    # an output laid out as the caller asks, nothing written beside it
    buf = torch.full((B, L, H, D + 8), 7.0, device="cuda")
    o = buf[..., :D].transpose(1, 2)
    got, _ = drl.dr_linear_attn_fwd(p["q"], p["k"], p["v"], p["la"], decay="head", o=o)
    assert got is o and (buf[..., D:] == 7).all()
    assert torch.equal(o, run_fwd(p, "head")[0])


@pytest.mark.parametrize("L", [1, 40, 100, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_row_for_every_token(L, dtype):
    """q, k, v and dO broadcast over tokens (stride 0), with a chunk that is not
    full: rows behind the last token must not count."""
    gen = torch.Generator().manual_seed(L)
    one = lambda n, D: torch.randn((2, n, 1, D), generator=gen).to(DT[dtype]).cuda().expand(2, n, L, D)  # noqa: E731
    p = dict(q=one(2, 64), k=one(2, 64), v=one(4, 72), dO=one(4, 72), la=decays(gen, "token", 2, 4, L),
             S0=torch.randn((2, 4, 64, 72), generator=gen).cuda(), dS=torch.randn((2, 4, 64, 72), generator=gen).cuda())
    check_fwd(p, "token")
    check_bwd(p, "token")
    # rows that overlap: each token's starts 8 channels after the last one's
    buf = torch.randn(8 * L + 64, generator=gen).to(DT[dtype]).cuda()
    p["q"] = p["k"] = buf.as_strided((2, 2, L, 64), (0, 0, 8, 1))
    check_fwd(p, "token")
    check_bwd(p, "token")


def test_offsets_past_32_bits():
    """Heads of q, k, v and o more than 2^31 elements apart."""
    gen = torch.Generator().manual_seed(4)
    L, D = 70, 64
    far = (1 << 31) + 64
    p = {}
    for n in ("q", "k", "v", "dO"):
        buf = torch.empty(far + L * D, dtype=torch.bfloat16, device="cuda")
        t = buf.as_strided((1, 2, L, D), (2 * far, far, D, 1))
        t.copy_(torch.randn((1, 2, L, D), generator=gen).cuda())
        p[n] = t
    p |= dict(la=decays(gen, "token", 1, 2, L), S0=None, dS=None)
    o = torch.empty(far + L * D, dtype=torch.float32, device="cuda").as_strided((1, 2, L, D), (2 * far, far, D, 1))
    check_fwd(p, "token", got=run_fwd(p, "token", o=o))
    small = {n: t.contiguous() if t is not None else None for n, t in p.items()}
    check_bwd(small, "token", got=run_bwd(p, "token"))


def test_a_bad_row_stays_in_its_sequence():
    p = problem(2, 2, 2, 130, 64, 64, "token", "bf16")
    clean, _ = run_fwd(p, "token")
    p["v"][0, 1, 70, 3] = math.nan
    p["k"][1, 0, 128, 0] = math.inf
    o, S = run_fwd(p, "token")
    assert torch.isnan(o[0, 1, 70, 3])
    assert torch.equal(o[0, 0], clean[0, 0]) and torch.equal(o[1, 1], clean[1, 1])
    assert torch.equal(o[0, 1, :64], clean[0, 1, :64]) and torch.equal(o[1, 0, :128], clean[1, 0, :128])


def test_same_bits_every_time_and_on_other_streams():
    p = problem(2, 4, 2, 700, 128, 64, "token", "bf16", grad=True)
    o, S = run_fwd(p, "token")
    g = run_bwd(p, "token")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    many = []
    for _ in range(3):
        for s in streams:   # calls in flight at once, each with what it allocates on its own stream
            many.append((run_fwd(p, "token", stream=s), run_bwd(p, "token", stream=s)))
    torch.cuda.synchronize()
    for (o2, S2), g2 in many:
        assert torch.equal(o, o2) and torch.equal(S, S2)
        assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("L,D,Hk,decay,dtype", [(1500, 64, 2, "token", "bf16"), (700, 128, 1, "head", "bf16"),
                                                (700, 128, 2, "token", "f32")])
def test_captured_and_replayed(L, D, Hk, decay, dtype):
    p = problem(1, 2, Hk, L, D, D, decay, dtype, grad=True)
    run_fwd(p, decay), run_bwd(p, decay)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = run_fwd(p, decay)
        g = run_bwd(p, decay)
    for n in range(4):
        gen = torch.Generator().manual_seed(100 + n)
        p["v"].copy_(torch.randn(p["v"].shape, generator=gen))
        p["S0"].copy_(torch.randn(p["S0"].shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        eo, eS = run_fwd(p, decay)
        eg = run_bwd(p, decay)
        assert torch.equal(o, eo) and torch.equal(S, eS)
        assert all(torch.equal(g[k], eg[k]) for k in g)


@pytest.mark.parametrize("decay", ["head", "token"])
def test_gradients_against_differences(decay):
    """Directional derivatives of <W, o> + <X, S_L> by central differences of
    the float64 forward, which at h = 2^-12 are off by h^2 / 6 times a third
    derivative: (q, k, v, S0) enter at most trilinearly and alpha as e^{h d},
    so 2^-26 of the terms' magnitude, next to the bound on the kernels' gradients."""
    p = problem(1, 4, 2, 90, 64, 64, decay, "f32", grad=True)
    g = run_bwd(p, decay)
    gen = torch.Generator().manual_seed(9)
    base = {n: p[n].double().cpu() for n in ("q", "k", "v", "la", "S0")}
    W, X = p["dO"].double().cpu(), p["dS"].double().cpu()

    def loss(t):
        H = t["v"].shape[1]
        B, L = t["v"].shape[0], t["v"].shape[2]
        o, S = ref.forward(ref.heads(t["q"], H), ref.heads(t["k"], H), t["v"], ref.gates(t["la"], decay, B, H, L), t["S0"])
        return float((W * o).sum() + (X * S).sum())

    names = {"q": "dq", "k": "dk", "v": "dv", "la": "dlog_alpha", "S0": "dS0"}
    _, size = ref.reference(p["q"], p["k"], p["v"], p["la"], p["S0"], decay, p["dO"], p["dS"])
    h = 2.0 ** -12
    for n, gn in names.items():
        d = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        plus, minus = ({**base, n: base[n] + s * h * d} for s in (1, -1))
        want = (loss(plus) - loss(minus)) / (2 * h)
        got = float((g[gn].double().cpu() * d).sum())
        bound = (ref.slack(90, 64, 64) + 2.0 ** -22) * float((size[gn] * d.abs()).sum())
        assert abs(got - want) <= bound, (n, got, want, bound)


def test_refusals_of_the_binding():
    import delta_rule_linear_amd as drl
    p = problem(1, 2, 2, 10, 64, 64, "token", "bf16")
    a = (p["q"], p["k"], p["v"])
    with pytest.raises(ValueError, match="decay"):
        drl.dr_linear_attn_fwd(*a, p["la"], decay="channel")
    with pytest.raises(ValueError, match="no log_alpha"):
        drl.dr_linear_attn_fwd(*a, p["la"], decay="none")
    with pytest.raises(ValueError, match="log_alpha has shape"):
        drl.dr_linear_attn_fwd(*a, p["la"], decay="head")
    with pytest.raises(TypeError):
        drl.dr_linear_attn_fwd(*a, None, decay="head")
    with pytest.raises(TypeError, match="k must be"):
        drl.dr_linear_attn_fwd(p["q"], p["k"].float(), p["v"], decay="none")
    with pytest.raises(ValueError, match="device tensor"):
        drl.dr_linear_attn_fwd(p["q"], p["k"].cpu(), p["v"], decay="none")
    with pytest.raises(ValueError, match="channels of a row"):
        drl.dr_linear_attn_fwd(p["q"], p["k"].transpose(2, 3).contiguous().transpose(2, 3), p["v"], decay="none")
    with pytest.raises(drl.DeltaRuleError, match="multiple of 16 bytes"):
        odd = torch.zeros(1, 2, 10, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
        drl.dr_linear_attn_fwd(odd, p["k"], p["v"], decay="none")
    with pytest.raises(drl.DeltaRuleError, match="not 16-byte aligned"):
        odd = torch.zeros(1, 2, 10, 72, dtype=torch.bfloat16, device="cuda")[..., 4:68]
        drl.dr_linear_attn_fwd(odd, p["k"], p["v"], decay="none")
    with pytest.raises(drl.DeltaRuleError, match="overlap"):
        o = torch.zeros(1, 1, 10, 64, device="cuda").expand(1, 2, 10, 64)
        drl.dr_linear_attn_fwd(*a, decay="none", o=o)
    with pytest.raises(drl.DeltaRuleError, match="overlaps"):
        drl.dr_linear_attn_fwd(*a, decay="none", o=p["v"], out_dtype=torch.bfloat16)
    with pytest.raises(drl.DeltaRuleError, match="workspace"):
        q = torch.zeros(1, 1, 4096, 64, dtype=torch.bfloat16, device="cuda")
        drl.dr_linear_attn_fwd(q, q, q, decay="none", workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="dO must be"):
        drl.dr_linear_attn_bwd(*a, None, None, p["v"].float(), decay="none")
