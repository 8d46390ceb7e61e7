"""The decay's gradient of the linear attention: configurations, its float64
value token by token, and a bound on what fp32 makes of it that a wrong
gradient does not pass.

    dlog_alpha_t = <S, dS>_E + sum over t <= s < E of (q_s . dq_s - k_s . dk_s)

with E the end of t's segment.  The sums themselves are fp64; what is off are
their terms.  An entry of dq_s (or S, dS) is a fp32 sum whose roundings are
relative to its partial sums, n = L + Dk + Dv + 256 of them at most (256 for the
decays' exponentials, as in linattn_ref), of either sign: a standard deviation
of sqrt(n) 2^-24 of the entry's usual size, the root mean square over its row
(or state).  Their sum weighted with q_s is off by that times |q_s| |dq_s| /
sqrt(Dk) where the errors are independent, and an error that a whole row shares
(a decay's) by that much of |q_s . dq_s|.  So one standard deviation is
sqrt(n) 2^-24 of

    T_s = |q_s . dq_s| + |k_s . dk_s| + (|q_s| |dq_s| + |k_s| |dk_s|) / sqrt(Dk)
    C_E = |<S, dS>_E| + |S| |dS| / sqrt(Dk Dv);

tokens share the states' errors, so T is added up and not its square.  Eight
standard deviations, and the result's own half step, are the bound.  All of it
is from the signed sums: no part grows with terms that the gradient does not
have."""
from __future__ import annotations

import math

import linattn_ref as ref
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# B, H, Hk, L, Dk, Dv, decay, dtype, lo, hi, resets, state, one row
CASES = [
    # lengths, heads, widths and types of the backward's other tests
    (1, 1, 1, 1, 64, 64, "token", "bf16", -0.1, -0.001, (), True, False),
    (2, 3, 3, 1, 128, 128, "head", "f32", -0.1, -0.001, (), True, False),
    (1, 2, 2, 63, 64, 64, "head", "bf16", -0.1, -0.001, (), True, False),
    (1, 2, 1, 64, 128, 128, "token", "bf16", -0.1, -0.001, (), True, False),
    (2, 2, 2, 65, 128, 64, "token", "bf16", -0.1, -0.001, (), True, False),
    (1, 6, 2, 130, 64, 96, "head", "bf16", -0.1, -0.001, (), True, False),
    (2, 4, 1, 200, 8, 8, "token", "bf16", -0.1, -0.001, (), True, False),
    (1, 3, 3, 200, 128, 8, "token", "f32", -0.1, -0.001, (), True, False),
    (1, 3, 1, 129, 48, 104, "token", "bf16", -0.1, -0.001, (), True, False),
    (1, 2, 2, 129, 72, 40, "head", "f32", -0.1, -0.001, (), True, False),
    (3, 5, 5, 192, 120, 24, "token", "bf16", -0.1, -0.001, (), True, False),
    (1, 4, 2, 90, 64, 64, "head", "f32", -0.1, -0.001, (), True, False),
    (1, 4, 2, 90, 64, 64, "token", "f32", -0.1, -0.001, (), True, False),
    (2, 2, 2, 100, 64, 64, "head", "bf16", -0.1, -0.001, (), False, False),
    (2, 2, 2, 100, 64, 64, "token", "bf16", -0.1, -0.001, (), False, False),
    # segments
    (1, 1, 1, 1000, 64, 32, "token", "bf16", -0.1, -0.001, (), True, False),
    (1, 2, 1, 1030, 128, 128, "head", "bf16", -0.1, -0.001, (), True, False),
    (1, 1, 1, 1100, 128, 128, "token", "f32", -0.1, -0.001, (), True, False),
    (1, 4, 2, 777, 64, 64, "token", "f32", -0.1, -0.001, (), True, False),
    (1, 1, 1, 4113, 128, 64, "token", "bf16", -0.02, 0.0, (), True, False),
    (1, 1, 1, 4113, 128, 64, "token", "f32", -0.02, 0.0, (), True, False),
    (1, 2, 1, 2500, 64, 128, "head", "bf16", -0.01, -0.0001, (), True, False),
    (1, 2, 1, 2500, 64, 128, "head", "f32", -0.01, -0.0001, (), True, False),
    # strong, absent and growing decays, and decays of zero
    *[(1, 2, 2, 300, 64, 64, "token", t, lo, hi, (), True, False) for t in ("bf16", "f32")
      for lo, hi in ((-3.0, -0.5), (-200.0, -1.0), (0.0, 0.0), (0.0, 0.02))],
    *[(1, 2, 1, 200, 64, 64, "token", t, -0.1, -0.001, (0, 64, 65, 131), True, False) for t in ("bf16", "f32")],
    # q, k, v and dO one row for all tokens
    *[(2, 4, 2, L, 64, 72, "token", t, -0.1, -0.001, (), True, True) for t in ("bf16", "f32") for L in (1, 40, 100, 700)],
    # so many sequences that each is one segment, of more than 1024 tokens
    *[(8, 64, 32, L, 8, 8, decay, t, -0.02, -0.0001, (), True, False)
      for L, decay, t in ((1025, "token", "bf16"), (1100, "head", "bf16"), (1100, "token", "f32"), (2100, "token", "bf16"),
                          (2100, "head", "f32"))],
]


def problem(B, H, Hk, L, Dk, Dv, decay, dtype, lo, hi, resets, state, one_row):
    """CPU tensors of a configuration."""
    gen = torch.Generator().manual_seed(L + Dk)
    n = 1 if one_row else L
    rows = lambda h, D, s=1.0: (s * torch.randn((B, h, n, D), generator=gen)).to(DT[dtype]).expand(B, h, L, D)  # noqa: E731
    p = dict(q=rows(Hk, Dk, Dk ** -0.5), k=rows(Hk, Dk), v=rows(H, Dv), dO=rows(H, Dv))
    p["la"] = lo + (hi - lo) * torch.rand((H,) if decay == "head" else (B, H, L), generator=gen)
    for t in resets:
        p["la"][:, :, t] = -math.inf
    for s in ("S0", "dS"):
        p[s] = torch.randn((B, H, Dk, Dv), generator=gen) if state else None
    return p


def segment_tokens(B, H, Hk, L, Dk, Dv):
    """Tokens per segment, from the size of the forward's workspace (a state and a
    decay for each segment)."""
    import delta_rule_linear_amd as drl
    need = drl.dr_linear_attn_fwd_workspace_bytes(drl.linattn_desc(B, H, Hk, L, Dk, Dv, drl.DR_BF16, drl.DR_F32, "token"))
    chunks = -(-L // 64)
    if need == 0:
        return 64 * chunks
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    nseg = next(s for s in range(2, chunks + 1) if up(B * H * s * Dk * Dv * 4) + up(B * H * s * 4) == need)
    return 64 * -(-chunks // nseg)


def reference(p, decay, seg):
    """dlog_alpha and its bound, per token [B, H, L], and the carries <S, dS> at
    the segments' ends [segments][B, H]."""
    d = lambda t: None if t is None else t.detach().double().cpu()  # noqa: E731
    q, k, v, S0, dO, dS = (d(p[n]) for n in ("q", "k", "v", "S0", "dO", "dS"))
    B, Hk, L, Dk = q.shape
    H, Dv = v.shape[1], v.shape[-1]
    q, k = ref.heads(q, H), ref.heads(k, H)
    a = ref.gates(p["la"], decay, B, H, L)
    dq, dk, _, dla, _ = ref.backward(q, k, v, a, S0, dO, dS)
    # the states at the segments' ends, S forwards and dS backwards
    ends = [min(L, e) for e in range(seg, L + seg, seg)]
    S = torch.zeros(B, H, Dk, Dv, dtype=torch.float64) if S0 is None else S0
    at = {}
    for t in range(L):
        S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        if t + 1 in ends:
            at[t + 1] = S
    G = torch.zeros(B, H, Dk, Dv, dtype=torch.float64) if dS is None else dS
    carry, spread = {}, {}
    for t in range(L, 0, -1):
        if t in at:
            s = at[t]
            carry[t] = (s * G).sum((-1, -2))
            spread[t] = carry[t].abs() + s.norm(dim=(-1, -2)) * G.norm(dim=(-1, -2)) * (Dk * Dv) ** -0.5
        G = a[:, :, t - 1, None, None] * (G + q[:, :, t - 1, :, None] * dO[:, :, t - 1, None, :])
    terms = sum((x * dx).sum(-1).abs() + x.norm(dim=-1) * dx.norm(dim=-1) * Dk ** -0.5 for x, dx in ((q, dq), (k, dk)))
    size = torch.empty_like(dla)
    for i, e in enumerate(ends):
        part = terms[:, :, i * seg:e]
        size[:, :, i * seg:e] = part.flip(-1).cumsum(-1).flip(-1) + spread[e][..., None]
    n = L + Dk + Dv + 256
    bound = 8 * n ** 0.5 * U * size + U * dla.abs() + ref.TINY
    return dict(dla=dla, bound=bound, carry=[carry[e] for e in ends], ends=ends, terms=(q * dq).sum(-1) - (k * dk).sum(-1))


def total(x, decay):
    """A gradient (or its bound) per token as the call returns it."""
    return x.sum((0, 2)) if decay == "head" else x


def check(got, r, decay):
    got, want, bound = got.detach().double().cpu(), total(r["dla"], decay), total(r["bound"], decay)
    assert got.shape == want.shape and bool(torch.isfinite(got).all())
    bad = (got - want).abs() / bound
    assert bool((bad <= 1).all()), f"dlog_alpha: {int((bad > 1).sum())} entries off, worst {float(bad.max()):.3g} of the bound"
    return float(bad.max())


def difference(p, decay, direction, h=2.0 ** -12):
    """The derivative of <dO, o> + <dS, S_L> along `direction` of log alpha, by
    differences of the float64 forward at h and 2 h, off by h^4 / 30 of a fifth
    derivative (2^-52) and 2^-52 / h of the loss's terms."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    B, H, L, _ = p["v"].shape
    q, k, v, S0, dO, dS = (d(p[n]) for n in ("q", "k", "v", "S0", "dO", "dS"))
    q, k = ref.heads(q, H), ref.heads(k, H)

    def loss(x):
        o, S = ref.forward(q, k, v, ref.gates(d(p["la"]) + x * direction, decay, B, H, L), S0)
        return float((dO * o).sum() + (dS * S).sum())

    return (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)


def check_difference(got, r, decay, direction, want):
    got = float((got.detach().double().cpu() * direction).sum())
    bound = float((total(r["bound"], decay) * direction.abs()).sum())
    assert abs(got - want) <= bound, f"off the differences: {got} instead of {want}, bound {bound:.3g}"
