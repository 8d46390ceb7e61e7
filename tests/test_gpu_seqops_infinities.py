"""Infinities and NaN on the GPU.  In the short convolution's backward they reach the
gradients that they are a part of, and no others.  In the gated recurrence an infinite state
stays infinite under every decay, wherever the sequence is cut into tiles."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seqops_ref as ref  # noqa: E402
from seqops_ref import DT, U, d, near  # noqa: E402

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def agree(got, want, bound, what):
    """The same infinities and NaN in the same places, and the others within the bound."""
    g = d(got)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what + ": NaN"
    ends = torch.isinf(want)
    assert torch.equal(torch.isinf(g), ends) and torch.equal(g[ends], want[ends]), what + ": infinities"
    ok = torch.isfinite(want)
    near(got.cpu()[ok], want[ok], bound.expand(want.shape)[ok], what)


# lengths that end on a step of the kernel's (a multiple of W, of four for two taps) and between two
@pytest.mark.parametrize("W,L", [(4, 8), (4, 9), (4, 64), (4, 259), (2, 8), (2, 7), (3, 12), (3, 13), (5, 51), (8, 16), (8, 85)])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("dtype,C", [("f32", 13), ("bf16", 16), ("bf16", 5)])
def test_convolution_backward(W, L, act, dtype, C):
    """One value that is infinite, or NaN, in the last tokens of a channel.  Tokens behind
    the last have no gradient, whatever the taps make of the rows before them."""
    import delta_rule_linear_amd as drl
    announce("convolution backward, infinities", W, L, act, dtype, C)
    gen = torch.Generator().manual_seed(W * 1000 + L)
    x = torch.randn((2, L, C), generator=gen).to(DT[dtype])
    dy = torch.randn((2, L, C), generator=gen).to(DT[dtype])
    w = torch.randn((C, W), generator=gen).abs() + 0.25
    w[:, 1::2] *= -1                                         # neighbouring taps of opposite signs
    b = torch.randn(C, generator=gen)
    clean = x.clone()
    for c, (back, v) in enumerate([(1, INF), (1, -INF), (1, NAN), (min(2, L), INF), (min(W, L), -INF)][:C]):
        x[0, L - back, c], clean[0, L - back, c] = v, 0.0
    g = drl.dr_short_conv_bwd(x.cuda(), w.cuda(), b.cuda(), None, dy.cuda(), activation=act, grad_dtype=torch.float32)
    x, clean, dy, w, b = (d(t) for t in (x, clean, dy, w, b))
    past = torch.cat([x.new_zeros(2, W - 1, C), x], 1)
    _, _, z = ref.conv_forward(x, w, b, None, False)
    # the slope of SiLU is 1 and 0 at the infinities
    zb = z.clamp(-1e4, 1e4)
    s = torch.sigmoid(zb)
    dz = dy * s * (1 + zb * (1 - s)) if act == "silu" else dy
    dz_err = torch.zeros_like(dz)
    if act == "silu":
        ez, _ = ref.conv_bounds(clean, w, b, None, True, ref.conv_forward(clean, w, b, None, True))
        dz_err = dy.abs() * (0.5 * ez + (12 + 4 * zb.abs()) * U * s * (1 + zb.abs() * (1 - s)))
        dz_err = torch.where(torch.isfinite(z), dz_err, 0 * dy)
    dx, mag, dw, bw = torch.zeros_like(past), torch.zeros_like(past), torch.zeros_like(w), torch.zeros_like(w)
    n = 2 * L + 8
    for j in range(W):
        dx[:, j:j + L] += w[:, j] * dz
        mag[:, j:j + L] += w[:, j].abs() * (dz_err + (W + 3) * U * dz.abs())
        dw[:, j] = (dz * past[:, j:j + L]).sum((0, 1))
        bw[:, j] = ((dz_err + n * U * dz.abs()) * past[:, j:j + L].abs()).sum((0, 1))
    agree(g["dx"], dx[:, W - 1:], mag[:, W - 1:], "dx")
    agree(g["dstate"], dx[:, :W - 1], mag[:, :W - 1], "dstate")
    agree(g["dweight"], dw, bw, "dweight")
    agree(g["dbias"], dz.sum((0, 1)), (dz_err + n * U * dz.abs()).sum((0, 1)), "dbias")


def decays(a, h):
    """a h, an infinite h kept under a decay of 0 as well; a NaN decay makes NaN of all."""
    return torch.where(torch.isinf(h) & ~torch.isnan(a), h, a * h)


def scan_forward(x, g, h0, decay, inputs):
    a, _, c = ref.scan_factors(g, decay, inputs)
    h, out = h0, []
    for t in range(x.shape[1]):
        h = decays(a[:, t], h) + c[:, t] * x[:, t]
        out.append(h)
    return torch.stack(out, 1), h


def finite(*ts):
    return [torch.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0) for t in ts]


def scan_case(B, L, C, decay, dtype, seed):
    """Gates of every strength, from none to resets, a memory of its own for each channel."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, dh = r(B, L, C).to(dtype), r(B, L, C).to(dtype)
    strength = torch.exp(torch.empty((B, 1, C)).uniform_(-9.0, 4.0, generator=gen))
    if decay == "log":
        g = -strength * torch.rand((B, L, C), generator=gen)
    else:
        g = -strength.log() + r(B, L, C)
    return x, g.to(dtype), r(B, C), dh, r(B, C), gen


def spoil(t, tokens, gen, values=(INF, -INF, NAN)):
    """Infinities and NaN at random places of a third of the channels, some channels with several."""
    B, L, C = t.shape
    for b in range(B):
        for c in range(0, C, 3):
            for _ in range(int(torch.randint(1, 4, (1,), generator=gen))):
                k = int(torch.randint(len(tokens), (1,), generator=gen))
                v = values[int(torch.randint(len(values), (1,), generator=gen))]
                t[b, min(tokens[k], L - 1), c] = v


# one token, runs of four, waves of 32, tiles of 128; many columns, which a workgroup walks, and few
SHAPES = [(1, 1, 9), (3, 3, 5), (2, 5, 64), (1, 33, 20), (2, 127, 16), (1, 130, 70), (2, 700, 33), (1, 3000, 65), (1100, 140, 7),
          (40, 300, 1700)]
TOKENS = [0, 1, 2, 3, 4, 5, 7, 8, 30, 31, 32, 33, 63, 95, 126, 127, 128, 129, 255, 256, 257, 500, 699, 1500, 2047, 2048, 2999]


@pytest.mark.parametrize("decay,inputs", [("log", "plain"), ("log", "blend"), ("logit", "unit"), ("logit", "plain")])
@pytest.mark.parametrize("B,L,C", SHAPES)
def test_recurrence(B, L, C, decay, inputs):
    import delta_rule_linear_amd as drl
    announce("recurrence, infinities", B, L, C, decay, inputs)
    x, g, h0, dh, dlast, gen = scan_case(B, L, C, decay, torch.float32, L + C)
    at = [t for t in TOKENS if t < L]
    some = slice(0, min(B, 2))   # what the reference sees of a batch: its first two sequences
    xs, h0s = x[some], h0[some]
    spoil(xs, at, gen)
    if C > 4:
        h0s[0, 1], h0s[0, 4] = INF, -INF
    if L > 2 and decay == "log":
        g[0, L // 2:, min(4, C - 1)] = -INF            # resets, and a long time of them
        g[0, L // 3, 0] = NAN
    m = dict(decay=decay, inputs=inputs)
    h, last = drl.dr_gated_scan_fwd(x.cuda(), g.cuda(), h0.cuda(), **m)
    args = d(xs), d(g[some]), d(h0s)
    want, wlast = scan_forward(*args, decay, inputs)
    e, elast = ref.scan_errors(*finite(args[0]), torch.nan_to_num(args[1], nan=0.0, neginf=-INF), *finite(args[2]), decay, inputs)
    agree(h[some], want, e, "h")
    agree(last[some], wlast, elast, "h_final")
    # the same token by token
    state = h0s.cuda()
    for t in range(min(L, 40)):
        y = drl.dr_gated_scan_step(state, xs[:, t].cuda().contiguous(), g[some][:, t].cuda().contiguous(), **m)
        agree(y, want[:, t], e[:, t], "h of a step")


@pytest.mark.parametrize("decay,inputs", [("log", "plain"), ("log", "blend"), ("logit", "unit"), ("logit", "plain")])
@pytest.mark.parametrize("B,L,C", SHAPES)
def test_recurrence_backward(B, L, C, decay, inputs):
    """Infinite and NaN gradients of h and of the last state: all that they are a part of is
    infinite or NaN, and the rest is as without them.  (Gates are below the strengths where
    products would be subnormal.)"""
    import delta_rule_linear_amd as drl
    announce("recurrence backward, infinities", B, L, C, decay, inputs)
    x, g, h0, dh, dlast, gen = scan_case(B, L, C, decay, torch.float32, L + C + 1)
    g = g.clamp(-30, 8)
    some = slice(0, min(B, 2))
    at = [L - 1 - t for t in TOKENS if t < L] + [t for t in TOKENS if t < L]
    dhs, dls = dh[some], dlast[some]
    spoil(dhs, at, gen)
    if C > 4:
        dls[0, 1], dls[0, 4] = INF, -INF
    m = dict(decay=decay, inputs=inputs)
    dev = [t.cuda() for t in (x, g, h0)]
    h, _ = drl.dr_gated_scan_fwd(*dev, **m)
    got = drl.dr_gated_scan_bwd(*dev, h, dh.cuda(), dlast.cuda(), **m)
    args = d(x[some]), d(g[some]), d(h0[some]), d(h[some])
    a, _, _ = ref.scan_factors(args[1], decay, inputs)
    e, D = d(dls), torch.empty_like(args[0])
    for t in range(L - 1, -1, -1):
        D[:, t] = d(dhs)[:, t] + e
        e = decays(a[:, t], D[:, t])
    clean = finite(d(dhs), d(dls))
    f = ref.scan_backward(*args, *clean, decay, inputs)
    ex, eg, e0 = ref.scan_back_errors(args[0], args[1], f, *clean, decay, inputs)
    for n, want, err in (("dx", f["c"] * D, ex), ("dgate", D * f["full"] * f["slope"], eg), ("dh0", e, e0)):
        v, ok = d(got[n][some]), torch.isfinite(want)
        assert torch.equal(torch.isfinite(v), ok), n
        near(got[n][some].cpu()[ok], want[ok], err[ok], n)


@pytest.mark.parametrize("L,C", [(200, 8), (5000, 8)])
def test_states_that_grow_out_of_range(L, C):
    """Sums that pass 2^128 become infinite and stay it; a forward that is cut in two agrees."""
    import delta_rule_linear_amd as drl
    x = torch.full((1, L, C), 2.0 ** 126, device="cuda")
    g = torch.zeros((1, L, C), device="cuda")
    g[0, :, 1] = -1.0                                        # stays below 2^127
    x[0, :, 2] *= -1
    h, last = drl.dr_gated_scan_fwd(x, g, None, decay="log")
    want, _ = scan_forward(d(x), d(g), torch.zeros(1, C, dtype=torch.float64), "log", "plain")
    want = torch.where(want.abs() >= 2.0 ** 128, want.sign() * INF, want)
    e, _ = ref.scan_errors(d(x), d(g), None, "log", "plain")
    agree(h, want, e, "h")
    assert torch.equal(last, h[:, -1])
    h1, s = drl.dr_gated_scan_fwd(x[:, :L // 3].contiguous(), g[:, :L // 3].contiguous(), None, decay="log")
    h2, _ = drl.dr_gated_scan_fwd(x[:, L // 3:].contiguous(), g[:, L // 3:].contiguous(), s, decay="log")
    agree(torch.cat([h1, h2], 1), want, e, "h in two parts")


@pytest.mark.parametrize("decay", ["log", "logit"])
@pytest.mark.parametrize("C", [6, 8, 200])
def test_recurrence_of_sixteen_bits_in_place_and_replayed(decay, C):
    """bf16 rows, NaN and infinite gates, the state carried in place, and a captured call
    whose inputs change between replays from clean to spoiled and back."""
    import delta_rule_linear_amd as drl
    L = 1300
    x, g, h0, _, _, gen = scan_case(1, L, C, decay, torch.bfloat16, C)
    clean = x.clone(), g.clone(), h0.clone()
    spoil(x, TOKENS, gen)
    g[0, 400, 1], g[0, 900, 2] = NAN, -INF
    if decay == "logit":
        g[0, 901:905, 2] = INF                       # a = 1
        g[0, 30, 4] = NAN
    h0[0, 5] = -INF
    m = dict(decay=decay, inputs="plain")
    dev = [t.cuda() for t in clean]
    graph = torch.cuda.CUDAGraph()
    drl.dr_gated_scan_fwd(*dev, **m)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        h, last = drl.dr_gated_scan_fwd(*dev, **m)
    for case in (clean, (x, g, h0), clean, (x, g, h0)):
        for t, v in zip(dev, case):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        args = tuple(d(v) for v in case)
        want, wlast = scan_forward(*args, decay, "plain")
        e, elast = ref.scan_errors(*finite(args[0]), torch.nan_to_num(args[1], nan=0.0, posinf=200.0, neginf=-INF if decay == "log" else -200.0),
                                   *finite(args[2]), decay, "plain")
        agree(h, want, e, "h")
        agree(last, wlast, elast, "h_final")
        s = dev[2].clone()
        h2, got = drl.dr_gated_scan_fwd(dev[0], dev[1], s, h_final=s, **m)
        assert got is s and torch.equal(torch.nan_to_num(h2, nan=7.0), torch.nan_to_num(h, nan=7.0))
        assert torch.equal(torch.nan_to_num(s, nan=7.0), torch.nan_to_num(last, nan=7.0))


@pytest.mark.parametrize("B,L,C", [(1, 9000, 130), (1, 700, 64), (600, 300, 70)])
@pytest.mark.parametrize("decay", ["log", "logit"])
def test_other_channels_keep_their_bits(B, L, C, decay):
    """Channels beside an infinite or NaN one, forward and backward, with memories that reach
    over many tiles."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(L)
    x, dh = torch.randn((B, L, C), generator=gen).cuda(), torch.randn((B, L, C), generator=gen).cuda()
    g = (-0.002 * torch.rand((B, L, C), generator=gen) if decay == "log" else 6 + torch.rand((B, L, C), generator=gen)).cuda()
    m = dict(decay=decay, inputs="blend")
    h, last = drl.dr_gated_scan_fwd(x, g, None, **m)
    base = drl.dr_gated_scan_bwd(x, g, None, h, dh, **m)
    y, dy = x.clone(), dh.clone()
    for c, v in ((3, INF), (20, NAN), (C - 1, -INF)):
        y[:, L // 3, c], dy[:, L // 2, c] = v, v
    h2, last2 = drl.dr_gated_scan_fwd(y, g, None, **m)
    back = drl.dr_gated_scan_bwd(x, g, None, h, dy, **m)
    keep = torch.ones(C, dtype=torch.bool, device="cuda")
    keep[[3, 20, C - 1]] = False
    assert torch.equal(h2[..., keep], h[..., keep]) and torch.equal(last2[:, keep], last[:, keep])
    assert torch.equal(h2[:, :L // 3], h[:, :L // 3]) and not torch.isfinite(h2[:, L // 3:, ~keep]).any()
    for n in ("dx", "dgate"):
        assert torch.equal(back[n][..., keep], base[n][..., keep]) and torch.equal(back[n][:, L // 2 + 1:], base[n][:, L // 2 + 1:])
    assert torch.equal(back["dh0"][:, keep], base["dh0"][:, keep])
