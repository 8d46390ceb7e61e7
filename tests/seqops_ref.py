"""The RMS norm, the short causal convolution and the gated linear recurrence in
float64 on the CPU, from their definitions, with the magnitudes that bound each
output's rounding (u = 2^-24 throughout)."""
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def d(t):
    return None if t is None else t.detach().double().cpu()


def near(got, want, bound, what):
    """got within `bound` of want, and half a step of its own type more."""
    half = {torch.bfloat16: 2.0 ** -8}.get(got.dtype, 0.0)
    got = d(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bound = bound + half * (want.abs() + bound) + 1e-37
    err = (got - want).abs()
    assert (err <= bound).all(), f"{what}: worst {float((err / bound).max()):.3g} of the bound"


# ---------------------------------------------------------------- RMS norm

def rms_forward(x, r, w, eps):
    """x [..., D], w [D] or shaped to broadcast: s, y, rstd."""
    s = x if r is None else x + r
    rstd = (s.square().mean(-1) + eps).rsqrt()
    y = s * rstd[..., None]
    return s, y if w is None else y * w, rstd


def rms_backward(s, w, rstd, dy, ds):
    n = s * rstd[..., None]
    t = dy if w is None else dy * w
    dx = rstd[..., None] * (t - n * (t * n).mean(-1, keepdim=True))
    return (dx if ds is None else dx + ds), dy * n


def e4m3_step(v):
    """The distance of e4m3 values around |v|."""
    return torch.exp2((torch.frexp(v)[1].clamp(min=-5) - 4).double())


# ---------------------------------------------------------------- convolution

def conv_forward(x, w, b, state, silu):
    B, L, C = x.shape
    W = w.shape[1]
    past = torch.cat([x.new_zeros(B, W - 1, C) if state is None else state, x], 1)
    z = x.new_zeros(B, L, C) if b is None else b.expand(B, L, C).clone()
    for t in range(L):
        for j in range(W):
            z[:, t] += w[:, j] * past[:, t + j]
    return (z * torch.sigmoid(z) if silu else z), past[:, L:], z


def conv_backward(x, w, b, state, dy, dlast, silu):
    B, L, C = x.shape
    W = w.shape[1]
    past = torch.cat([x.new_zeros(B, W - 1, C) if state is None else state, x], 1)
    _, _, z = conv_forward(x, w, b, state, silu)
    s = torch.sigmoid(z)
    dz = dy * s * (1 + z * (1 - s)) if silu else dy
    dp = torch.zeros_like(past)
    dw = torch.zeros_like(w)
    for j in range(W):
        dp[:, j:j + L] += w[:, j] * dz
        dw[:, j] = (dz * past[:, j:j + L]).sum((0, 1))
    if dlast is not None:
        dp[:, L:] += dlast
    return {"dx": dp[:, W - 1:], "dstate": dp[:, :W - 1], "dweight": dw, "dbias": dz.sum((0, 1)), "dz": dz, "z": z,
            "past": past}


def conv_bounds(x, w, b, state, silu, out):
    """Of z and y: W + 1 terms, each rounded once or twice; SiLU's slope is below 1.1,
    its sigmoid off by the exponent's 2 |z| u (times 1 - s) and a few u more."""
    W = w.shape[1]
    _, _, mag = conv_forward(x.abs(), w.abs(), None if b is None else b.abs(), None if state is None else state.abs(), False)
    dz = (W + 2) * U * mag
    if not silu:
        return dz, dz
    y, _, z = out
    s = torch.sigmoid(z)
    return dz, 1.1 * dz + y.abs() * (8 + 3 * z.abs() * (1 - s)) * U


# ---------------------------------------------------------------- recurrence

def scan_factors(g, decay, inputs):
    if decay == "log":
        a, rest = g.exp(), -torch.expm1(g)
    else:
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    c = {"plain": torch.ones_like(a), "blend": rest, "unit": (rest * (1 + a)).sqrt()}[inputs]
    return a, rest, c


def scan_forward(x, g, h0, decay, inputs):
    a, _, c = scan_factors(g, decay, inputs)
    h = x.new_zeros(x.shape[0], x.shape[2]) if h0 is None else h0
    out = []
    for t in range(x.shape[1]):
        h = a[:, t] * h + c[:, t] * x[:, t]
        out.append(h)
    return torch.stack(out, 1) if out else torch.empty_like(x), h


def scan_backward(x, g, h0, h, dh, dlast, decay, inputs):
    """The gradients from the kept h; also d, the sums that bound its rounding."""
    a, rest, c = scan_factors(g, decay, inputs)
    B, L, C = x.shape
    e = x.new_zeros(B, C) if dlast is None else dlast
    mag = e.abs()
    D, M = torch.empty_like(x), torch.empty_like(x)
    for t in range(L - 1, -1, -1):
        D[:, t], M[:, t] = dh[:, t] + e, dh[:, t].abs() + mag
        e, mag = a[:, t] * D[:, t], a[:, t] * M[:, t]
    before = torch.cat([x.new_zeros(B, 1, C) if h0 is None else h0[:, None], h[:, :-1]], 1)
    if inputs == "blend":
        full, size = before - x, before.abs() + x.abs()
    elif inputs == "unit":
        k = torch.where(c > 0, a / c, torch.zeros_like(c))
        full, size = before - k * x, before.abs() + (k * x).abs()
    else:
        full, size = before, before.abs()
    slope = a if decay == "log" else a * rest
    return {"dx": c * D, "dgate": D * full * slope, "dh0": e, "D": D, "M": M, "full": full, "size": size, "slope": slope,
            "c": c}


def decay_bound(g, a, rest):
    """The kernels' a: 1 - a is off by (2 |g| + 6) u of itself where a > 1/2, a by as
    much of itself below about 2/3; the smaller of the two at most doubles between.  A
    state that grows (a > 1) has a rounded to fp32, off by (2 |g| + 4) u of itself."""
    size = (4 * torch.nan_to_num(g, neginf=0.0).abs() + 12) * U
    return size * torch.where(rest < 0, a, torch.minimum(a, rest))


def scan_errors(x, g, h0, decay, inputs):
    """What h may be off by: every step rounds a few times, relative to the sum of
    absolute values M, and a and c are off by decay_bound and (2 |g| + 10) u."""
    a, rest, c = scan_factors(g, decay, inputs)
    ga = torch.nan_to_num(g, neginf=0.0).abs()
    da, dc = decay_bound(g, a, rest), c.abs() * (2 * ga + 10) * U * (inputs != "plain")
    B, L, C = x.shape
    M = x.new_zeros(B, C) if h0 is None else h0.abs()
    E = torch.zeros_like(M)
    out = torch.empty_like(x)
    for t in range(L):
        before = M
        M = a[:, t] * M + (c[:, t] * x[:, t]).abs()
        grows = (rest[:, t] < 0) * (inputs != "plain") * 8 * U   # 1 - a from e^g
        E = a[:, t] * E + da[:, t] * before + (dc[:, t] + grows) * x[:, t].abs() + 8 * U * M
        out[:, t] = E
    return out, E


def scan_back_errors(x, g, ref, dh, dlast, decay, inputs):
    """The same for d; dx and dgate are products of it."""
    a, rest, c = scan_factors(g, decay, inputs)
    ga = torch.nan_to_num(g, neginf=0.0).abs()
    da = decay_bound(g, a, rest)
    E = torch.zeros_like(x[:, 0])
    ED = torch.empty_like(x)
    for t in range(x.shape[1] - 1, -1, -1):
        ED[:, t] = E + 8 * U * ref["M"][:, t]
        E = a[:, t] * ED[:, t] + da[:, t] * ref["M"][:, t] + 8 * U * a[:, t] * ref["M"][:, t]
    rel = (2 * ga + 12) * U
    # where the state grows, 1 - a comes from e^g and is off by fp32's rounding of that
    dx = c.abs() * ED + (c.abs() * rel + torch.where(rest < 0, rel, 0 * rel)) * ref["D"].abs()
    dg = ref["slope"] * (ED * ref["full"].abs() + ref["M"] * ref["size"] * (2 * rel + 4 * U))
    return dx, dg, E
