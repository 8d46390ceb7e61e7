"""Linear attention with a decay per head and layer norm in float64 on the CPU,
token by token, and the magnitudes that bound the rounding of a float32
computation: the same sums with every term's absolute value.

Bounds.  A float32 sum of n terms is off by at most n 2^-24 of the sum of the
terms' absolute values, whatever its order (and by about sqrt(n) 2^-24 where the
roundings are independent).  An output entry is such a sum over the channels of
a contraction, the tokens before it and S0, so n = L + Dk + Dv; 256 more cover
the decays' exponentials (a few roundings each, and the rounding of an
exponent u <= 128 that 2^-u scales).  bf16 outputs add their own half step, 2^-8
of the value, and, where the products carry fp32 values in two bf16 terms, 2^-16
of the magnitude (two half steps of 2^-8)."""
from __future__ import annotations

import torch

TINY = 1e-30   # results that underflow float32


def slack(L, Dk, Dv):
    return (L + Dk + Dv + 256) * 2.0 ** -24


def heads(x, H):
    return x.repeat_interleave(H // x.shape[1], dim=1)


def gates(la, decay, B, H, L):
    if decay == "none":
        return torch.ones(B, H, L, dtype=torch.float64)
    a = la.double().cpu().exp()
    return a[None, :, None].expand(B, H, L) if decay == "head" else a


def forward(q, k, v, a, S0=None):
    """q, k, v [B,H,L,D], a [B,H,L] in float64: o, S_L."""
    B, H, L, Dk = q.shape
    Dv = v.shape[-1]
    S = torch.zeros(B, H, Dk, Dv, dtype=torch.float64) if S0 is None else S0.clone()
    o = torch.empty(B, H, L, Dv, dtype=torch.float64)
    for t in range(L):
        S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, t] = (S * q[:, :, t, :, None]).sum(-2)
    return o, S


def backward(q, k, v, a, S0, dO, dS):
    """Gradients by the formulas, with one q and k head per state head:
    dq, dk, dv, dla [B,H,L], dS0."""
    B, H, L, Dk = q.shape
    Dv = v.shape[-1]
    S = torch.zeros(B, H, Dk, Dv, dtype=torch.float64) if S0 is None else S0.clone()
    before = []
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dla = torch.empty(B, H, L, dtype=torch.float64)
    for t in range(L):
        before.append(S)
        S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        dq[:, :, t] = (S * dO[:, :, t, None, :]).sum(-1)
    G = torch.zeros_like(S) if dS is None else dS.clone()
    for t in range(L - 1, -1, -1):
        G = G + q[:, :, t, :, None] * dO[:, :, t, None, :]
        dk[:, :, t] = (G * v[:, :, t, None, :]).sum(-1)
        dv[:, :, t] = (G * k[:, :, t, :, None]).sum(-2)
        dla[:, :, t] = a[:, :, t] * (before[t] * G).sum((-1, -2))
        G = a[:, :, t, None, None] * G
    return dq, dk, dv, dla, G


def shared(dx, Hk):
    B, H = dx.shape[:2]
    return dx.reshape(B, Hk, H // Hk, *dx.shape[2:]).sum(2)


def reference(q, k, v, la, S0, decay, dO=None, dS=None):
    """What dr_linear_attn_fwd (and _bwd, with dO) returns, and the magnitudes
    of its entries, as two dicts of float64 CPU tensors."""
    d = lambda t: None if t is None else t.detach().double().cpu()  # noqa: E731
    q, k, v, S0, dO, dS = (d(t) for t in (q, k, v, S0, dO, dS))
    B, Hk, L, Dk = q.shape
    H = v.shape[1]
    a = gates(la, decay, B, H, L)
    out = []
    for fn in (lambda t: t, lambda t: None if t is None else t.abs()):
        Q, K, V, Z = heads(fn(q), H), heads(fn(k), H), fn(v), fn(S0)
        o, S = forward(Q, K, V, a, Z)
        r = {"o": o, "S": S}
        if dO is not None:
            dq, dk, dv, dla, dS0 = backward(Q, K, V, a, Z, fn(dO), fn(dS))
            if out:   # magnitudes: the sums that d log alpha is taken from
                tail = ((Q * dq).sum(-1) + (K * dk).sum(-1)).sum(-1, keepdim=True)
                end = 0 if dS is None else (S * fn(dS)).sum((-1, -2))[..., None]
                dla = (tail + end).expand(B, H, L)
            r |= {"dq": shared(dq, Hk), "dk": shared(dk, Hk), "dv": dv, "dS0": dS0,
                  "dlog_alpha": dla.sum((0, 2)) if decay == "head" else dla}
        out.append(r)
    return out


def check(got, want, size, n, what, bf16=False, two_terms=True):
    """Every entry within the worst case, and the whole within the expected
    size (8 standard deviations' worth) of the roundings of n-term sums."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: not finite"
    err = (got - want).abs()
    step = 2.0 ** -8 * want.abs() + (2.0 ** -16 * size if two_terms else 0) if bf16 else 0
    worst = n * size + step + TINY
    bad = err > worst
    assert not bad.any(), f"{what}: {int(bad.sum())} entries off, worst {float((err / worst).max()):.3g} of the bound"
    if got.numel():
        terms = n * 2.0 ** 24
        bound = 8 * terms ** 0.5 * 2.0 ** -24 * float(size.norm()) + TINY
        if bf16:
            bound += 2.0 ** -8 * float(want.norm()) + 2.0 ** -16 * float(size.norm())
        assert float(err.norm()) <= bound, f"{what}: 2-norm of the error {float(err.norm()):.3g}, bound {bound:.3g}"


def norm_forward(x, w, b, eps):
    """x [B,H,L,D], w and b [D] or [H,D] (or None), float64."""
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    wide = lambda t: t[None, :, None] if t.dim() == 2 else t  # noqa: E731
    y = (x - mean) * rstd
    y = y if w is None else y * wide(w)
    y = y if b is None else y + wide(b)
    return y, mean[..., 0], rstd[..., 0]


def norm_backward(x, w, mean, rstd, dy, per_head):
    n = (x - mean[..., None]) * rstd[..., None]
    t = dy if w is None else dy * (w[None, :, None] if w.dim() == 2 else w)
    dx = rstd[..., None] * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    over = (0, 2) if per_head else (0, 1, 2)
    return dx, (dy * n).sum(over), dy.sum(over)
