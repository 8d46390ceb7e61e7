"""Linear attention with a decay for each head (chunked forward, its backward, one-token step)
and the layer norm of its output (forward and backward): the cases to measure, their inputs,
their plain forms in elementary torch operations, and their values in 64 bits.

    S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t        a_t = e^{log_alpha}
    y = (x - mean) / sqrt(var + eps) * weight + bias
"""
import math

import torch

own = False

CHUNK = 128   # tokens per chunk of the plain form
EPS = 1e-5

BF16, F32 = "bf16", "f32"


def _fwd(name, B, H, Hk, L, Dk, Dv, decay, dtype, out, token_major=False, state=True):
    return {"name": name, "op": "fwd", "B": B, "H": H, "Hk": Hk, "L": L, "Dk": Dk, "Dv": Dv, "decay": decay,
            "dtype": dtype, "out": out, "token_major": token_major, "state": state}


def _bwd(name, B, H, Hk, L, Dk, Dv, decay, dtype, out, token_major=False, state=True):
    return {**_fwd(name, B, H, Hk, L, Dk, Dv, decay, dtype, out, token_major, state), "op": "bwd"}


def _step(name, N, H, Hk, Dk, Dv, decay, dtype, out):
    return {"name": name, "op": "step", "N": N, "H": H, "Hk": Hk, "Dk": Dk, "Dv": Dv, "decay": decay,
            "dtype": dtype, "out": out}


def _norm(name, op, B, H, L, D, per_head, dtype, out, token_major=False):
    return {"name": name, "op": op, "B": B, "H": H, "L": L, "D": D, "per_head": per_head, "dtype": dtype,
            "out": out, "token_major": token_major}


def listed():
    return [
        # a training or prefill batch of long sequences, the shape of the repository's own long-prefill benchmark
        _fwd("fwd long", 2, 16, 16, 16384, 128, 128, "token", BF16, BF16),
        # a short prompt of odd length with one constant decay per head; latency counts
        _fwd("fwd short prompt", 1, 16, 16, 77, 64, 64, "head", BF16, F32),
        # many sequences that share q and k heads among four state heads, rows as a projection leaves them
        _fwd("fwd shared heads", 16, 32, 8, 2000, 128, 64, "token", BF16, BF16, token_major=True),
        # fp32 inputs at the size of the repository's fp32 chunked benchmark
        _fwd("fwd fp32", 1, 16, 16, 4096, 128, 128, "head", F32, F32),
        # training at the long shape
        _bwd("bwd long", 2, 16, 16, 16384, 128, 128, "token", BF16, BF16),
        # training on a small batch of odd length, shared heads, unequal head sizes, gradients kept in 32 bits
        _bwd("bwd ragged", 3, 12, 4, 1111, 64, 96, "head", BF16, F32),
        # one conversation's next token
        _step("step one", 1, 16, 16, 128, 128, "head", BF16, BF16),
        # the repository's decode batch
        _step("step batch", 256, 16, 16, 128, 128, "token", BF16, F32),
        # the per-head norm of the long forward's output, written token-major for the output projection
        _norm("norm fwd heads", "norm_fwd", 2, 16, 16384, 128, True, BF16, BF16, token_major=True),
        # a few rows of an odd width in fp32
        _norm("norm fwd odd", "norm_fwd", 1, 1, 300, 1001, False, F32, F32),
        # the per-head norm's backward at the long shape
        _norm("norm bwd heads", "norm_bwd", 2, 16, 16384, 128, True, BF16, BF16, token_major=True),
        # a block's norm over the model width, one weight for all rows
        _norm("norm bwd width", "norm_bwd", 1, 1, 8191, 2048, False, BF16, BF16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd"))
    dtype = rng.choice((BF16, BF16, BF16, F32))
    out = F32 if dtype == F32 else rng.choice((BF16, F32))
    dims = (64, 128, 64, 128, 8 * rng.randint(2, 16))
    decay = rng.choice(("token", "head", "token", "head", "none"))
    Hk = rng.choice((1, 2, 4, 8, 16, 3))
    H = Hk * rng.choice((1, 1, 1, 2, 4))
    if op in ("fwd", "bwd"):
        L = _log_int(rng, 1, 16384)
        most = 524288 if dtype == BF16 else 65536
        B = _log_int(rng, 1, max(1, min(64, most // (H * L))))
        if B * H * L > most:
            L = most // (B * H)
        mk = _fwd if op == "fwd" else _bwd
        case = mk("", B, H, Hk, L, rng.choice(dims), rng.choice(dims), decay, dtype, out,
                  token_major=rng.random() < 0.5, state=rng.random() < 0.7)
    elif op == "step":
        case = _step("", _log_int(rng, 1, max(1, 4096 // H)), H, Hk, rng.choice(dims), rng.choice(dims), decay, dtype, out)
    elif rng.random() < 0.5:
        L = _log_int(rng, 1, 16384)
        case = _norm("", op, _log_int(rng, 1, max(1, 524288 // (H * L))), H, L, rng.choice((64, 128, rng.randint(3, 256))),
                     True, dtype, out, token_major=rng.random() < 0.5)
        if case["B"] * H * L * case["D"] > 524288 * 128:
            case["L"] = max(1, 524288 * 128 // (case["B"] * H * case["D"]))
    else:
        D = _log_int(rng, 1, 8192)
        case = _norm("", op, 1, 1, _log_int(rng, 1, 524288 * 128 // max(D, 128)), D, False, dtype, out)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _type(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _rows(gen, shape, token_major, dtype, unit=False):
    """A [B, H, L, D] tensor; token-major: a view of [B, L, H, D], as a projection writes it."""
    B, H, L, D = shape
    x = torch.randn((B, L, H, D) if token_major else shape, device="cuda", generator=gen)
    x = (_unit(x) if unit else x).to(_type(dtype))
    return x.transpose(1, 2) if token_major else x


def _decays(gen, decay, lead, H):
    """Constant decays 1 - 2^-5 ... 1 - 2^-12 over the heads, or one draw per token in [-0.1, -0.001]."""
    if decay == "none":
        return None
    if decay == "head":
        e = torch.linspace(-5, -12, H, device="cuda")
        jitter = torch.rand(H, device="cuda", generator=gen) * 0.1
        return torch.log1p(-torch.exp2(e + jitter))
    return -(0.001 + 0.099 * torch.rand(lead, device="cuda", generator=gen))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    s = {"case": dict(c)}
    if c["op"] in ("fwd", "bwd"):
        B, H, Hk, L, Dk, Dv = (c[n] for n in ("B", "H", "Hk", "L", "Dk", "Dv"))
        tm, dt = c["token_major"], c["dtype"]
        s["q"] = _rows(gen, (B, Hk, L, Dk), tm, dt, True)
        s["k"] = _rows(gen, (B, Hk, L, Dk), tm, dt, True)
        s["v"] = _rows(gen, (B, H, L, Dv), tm, dt)
        s["la"] = _decays(gen, c["decay"], (B, H, L), H)
        s["S0"] = 0.1 * torch.randn((B, H, Dk, Dv), device="cuda", generator=gen) if c["state"] else None
        if c["op"] == "bwd":
            s["dO"] = _rows(gen, (B, H, L, Dv), tm, dt)
            s["dS"] = torch.randn((B, H, Dk, Dv), device="cuda", generator=gen) if c["state"] else None
    elif c["op"] == "step":
        N, H, Hk, Dk, Dv = (c[n] for n in ("N", "H", "Hk", "Dk", "Dv"))
        s["S"] = 0.1 * torch.randn((N, H, Dk, Dv), device="cuda", generator=gen)
        s["q"] = _unit(torch.randn((N, Hk, Dk), device="cuda", generator=gen)).to(_type(c["dtype"]))
        s["k"] = _unit(torch.randn((N, Hk, Dk), device="cuda", generator=gen)).to(_type(c["dtype"]))
        s["v"] = torch.randn((N, H, Dv), device="cuda", generator=gen).to(_type(c["dtype"]))
        s["la"] = _decays(gen, c["decay"], (N, H), H)
    else:
        B, H, L, D = (c[n] for n in ("B", "H", "L", "D"))
        s["x"] = (0.3 + torch.randn((B, H, L, D), device="cuda", generator=gen)).to(_type(c["dtype"]))
        wshape = (H, D) if c["per_head"] else (D,)
        s["w"] = 1 + 0.1 * torch.randn(wshape, device="cuda", generator=gen)
        s["b"] = 0.1 * torch.randn(wshape, device="cuda", generator=gen)
        if c["op"] == "norm_fwd" and c["token_major"]:
            # the output rows in the order that the output projection reads
            s["y"] = torch.empty((B, L, H, D), device="cuda", dtype=_type(c["out"])).transpose(1, 2)
        if c["op"] == "norm_bwd":
            s["dy"] = _rows(gen, (B, H, L, D), c["token_major"], c["dtype"])
            x = s["x"].double()
            mean = x.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[..., None]).square().mean(-1) + EPS).rsqrt().float()
    return s


# ---------------------------------------------------------------- plain forms

def _heads(x, H):
    """q or k with every state head's own copy, in fp32."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _shared(dx, Hk):
    """The sum of a gradient over the state heads that share a q or k head."""
    B, H = dx.shape[:2]
    return dx.reshape(B, Hk, H // Hk, *dx.shape[2:]).sum(2)


def _gate(la, case, lead):
    if la is None:
        return torch.zeros(lead, device="cuda", dtype=torch.float64)
    g = la.double()
    return g[None, :, None].expand(lead) if case["decay"] == "head" else g


def _chunks(x, n):
    B, H, L = x.shape[:3]
    pad = x.new_zeros((B, H, n * CHUNK - L) + tuple(x.shape[3:]))
    return torch.cat([x, pad], 2).reshape((B, H, n, CHUNK) + tuple(x.shape[3:]))


def _attend(x, y, z, la, start, inclusive=True):
    """out_i = sum_{j <= i} e^{u_i - u_j} (x_i . y_j) z_j + e^{u_i} start^T x_i and the state after the
    last token, u the running sum of la (with or without the row's own). Chunk by chunk: products within a
    chunk, and one triangular product over the chunks' states. fp32, the running sums in 64 bits."""
    B, H, L, Dx = x.shape
    Dz = z.shape[-1]
    n = -(-L // CHUNK)
    x, y, z, la = (_chunks(t, n) for t in (x, y, z, la))
    s = la.cumsum(-1)
    u, total = (s if inclusive else s - la), s[..., -1:]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    pair = torch.where(low, u[..., :, None] - u[..., None, :], -math.inf).exp().float()
    inner = y * (total - u).exp().float()[..., None]
    local = torch.matmul(inner.transpose(-1, -2), z).reshape(B, H, n, Dx * Dz)
    first = start.reshape(B, H, 1, Dx * Dz) if start is not None else local.new_zeros(B, H, 1, Dx * Dz)
    ends = torch.cat([torch.zeros_like(total[:, :, :1, 0]), total[..., 0].cumsum(-1)], -1)
    low = torch.ones(n + 1, n + 1, dtype=torch.bool, device="cuda").tril()
    across = torch.where(low, ends[..., :, None] - ends[..., None, :], -math.inf).exp().float()
    states = torch.matmul(across, torch.cat([first, local], 2)).reshape(B, H, n + 1, Dx, Dz)
    out = torch.matmul(x, states[:, :, :n]) * u.exp().float()[..., None]
    out = out + torch.matmul(torch.matmul(x, y.transpose(-1, -2)) * pair, z)
    return out.reshape(B, H, n * CHUNK, Dz)[:, :, :L], states[:, :, n]


def _plain_fwd(s):
    c = s["case"]
    B, H, L = c["B"], c["H"], c["L"]
    o, S = _attend(_heads(s["q"], H), _heads(s["k"], H), s["v"].float(), _gate(s["la"], c, (B, H, L)), s["S0"])
    return o.to(_type(c["out"])), S.contiguous()


def _plain_bwd(s):
    c = s["case"]
    B, H, Hk, L, Dk, Dv = (c[n] for n in ("B", "H", "Hk", "L", "Dk", "Dv"))
    q, k, v, dO = _heads(s["q"], H), _heads(s["k"], H), s["v"].float(), s["dO"].float()
    la = _gate(s["la"], c, (B, H, L))
    back = [t.flip(2) for t in (q, k, v, dO, la)]
    dq, St = _attend(dO, v, k, la, None if s["S0"] is None else s["S0"].transpose(-1, -2))
    dS = s["dS"]
    dv, dS0 = _attend(back[1], back[0], back[3], back[4], dS, inclusive=False)
    dk, _ = _attend(back[2], back[3], back[0], back[4], None if dS is None else dS.transpose(-1, -2), inclusive=False)
    dk, dv = dk.flip(2), dv.flip(2)
    to = _type(c["out"])
    out = {"dq": _shared(dq, Hk).to(to), "dk": _shared(dk, Hk).to(to), "dv": dv.to(to),
           "dS0": dS0.contiguous(), "dlog_alpha": None}
    if c["decay"] != "none":
        # d log alpha_t = <S_L, dS_L> + sum over s >= t of q_s . dq_s - k_s . dk_s: long sums in 64 bits
        d = ((q * dq).sum(-1) - (k * dk).sum(-1)).double()
        tail = d.flip(-1).cumsum(-1).flip(-1)
        if dS is not None:
            tail = tail + (St.transpose(-1, -2).double() * dS.double()).sum((-1, -2))[..., None]
        out["dlog_alpha"] = (tail if c["decay"] == "token" else tail.sum((0, 2))).float()
    return out


def _plain_step(s):
    c = s["case"]
    g = c["H"] // c["Hk"]
    q, k = (s[n].float().repeat_interleave(g, dim=1) for n in ("q", "k"))
    S = s["S"]
    if s["la"] is not None:
        a = s["la"].exp()
        S.mul_(a[None, :, None, None] if c["decay"] == "head" else a[..., None, None])
    S.add_(k[..., :, None] * s["v"].float()[..., None, :])
    o = (S * q[..., :, None]).sum(-2)
    return o.to(_type(c["out"])), S


def _wide(w, case):
    return w[None, :, None, :] if case["per_head"] else w


def _plain_norm_fwd(s):
    c = s["case"]
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = (d * rstd * _wide(s["w"], c) + _wide(s["b"], c)).to(_type(c["out"]))
    if "y" in s:
        y = s["y"].copy_(y)
    return y, mean[..., 0], rstd[..., 0]


def _plain_norm_bwd(s):
    c = s["case"]
    dy, r = s["dy"].float(), s["rstd"][..., None]
    xh = (s["x"].float() - s["mean"][..., None]) * r
    t = dy * _wide(s["w"], c)
    dx = r * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    over = (0, 2) if c["per_head"] else (0, 1, 2)
    return {"dx": dx.to(_type(c["out"])), "dweight": (dy * xh).sum(over), "dbias": dy.sum(over)}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd}[op](s)
    import delta_rule_linear_amd as drl
    to = _type(c["out"])
    if op == "fwd":
        return drl.dr_linear_attn_fwd(s["q"], s["k"], s["v"], s["la"], s["S0"], decay=c["decay"], out_dtype=to)
    if op == "bwd":
        return drl.dr_linear_attn_bwd(s["q"], s["k"], s["v"], s["la"], s["S0"], s["dO"], s["dS"], decay=c["decay"],
                                      grad_dtype=to)
    if op == "step":
        return drl.dr_linear_attn_step(s["S"], s["q"], s["k"], s["v"], s["la"], decay=c["decay"], out_dtype=to), s["S"]
    if op == "norm_fwd":
        return drl.dr_layernorm_fwd(s["x"], s["w"], s["b"], eps=EPS, out_dtype=to, y=s.get("y"))
    return drl.dr_layernorm_bwd(s["x"], s["w"], s["mean"], s["rstd"], s["dy"], grad_dtype=to)


def work(case):
    c = case
    size = {BF16: 2, F32: 4}
    i, o = size[c["dtype"]], size[c["out"]]
    if c["op"] in ("fwd", "bwd"):
        T, Tk = c["B"] * c["H"] * c["L"], c["B"] * c["Hk"] * c["L"]
        Dk, Dv = c["Dk"], c["Dv"]
        S = 4 * c["B"] * c["H"] * Dk * Dv
        la = {"none": 0, "head": 4 * c["H"], "token": 4 * T}[c["decay"]]
        ins = i * (2 * Tk * Dk + T * Dv) + la + (S if c["state"] else 0)
        if c["op"] == "fwd":
            return {"bytes": ins + o * T * Dv + S, "flops": 4 * T * Dk * Dv}
        return {"bytes": ins + i * T * Dv + (S if c["state"] else 0) + o * (2 * Tk * Dk + T * Dv) + la + S,
                "flops": 10 * T * Dk * Dv}
    if c["op"] == "step":
        T, Dk, Dv = c["N"] * c["H"], c["Dk"], c["Dv"]
        la = {"none": 0, "head": 4 * c["H"], "token": 4 * T}[c["decay"]]
        return {"bytes": 8 * T * Dk * Dv + i * (2 * c["N"] * c["Hk"] * Dk + T * Dv) + o * T * Dv + la,
                "flops": 5 * T * Dk * Dv}
    rows, D = c["B"] * c["H"] * c["L"], c["D"]
    w = 8 * D * (c["H"] if c["per_head"] else 1)
    if c["op"] == "norm_fwd":
        return {"bytes": rows * (D * (i + o) + 8) + w, "flops": 8 * rows * D}
    return {"bytes": rows * (D * (2 * i + o) + 8) + w // 2 + w, "flops": 14 * rows * D}


# ---------------------------------------------------------------- in 64 bits, token by token

def _exact_attention(case, seed):
    c, s = case, prepare(case, seed)
    B, H, Hk, L, Dk, Dv = (c[n] for n in ("B", "H", "Hk", "L", "Dk", "Dv"))
    rep = torch.arange(H, device="cuda") // (H // Hk)
    by_token = lambda t: t.double().permute(2, 0, 1, 3).contiguous()  # noqa: E731
    q, k, v = by_token(s["q"][:, rep]), by_token(s["k"][:, rep]), by_token(s["v"])
    if s["la"] is None:
        a = torch.ones(L, B, H, device="cuda", dtype=torch.float64)
    elif c["decay"] == "head":
        a = s["la"].double().exp().expand(L, B, H).contiguous()
    else:
        a = s["la"].double().exp().permute(2, 0, 1).contiguous()
    zero = torch.zeros(B, H, Dk, Dv, device="cuda", dtype=torch.float64)
    S = zero.clone() if s["S0"] is None else s["S0"].double()
    if c["op"] == "fwd":
        o = torch.empty(L, B, H, Dv, device="cuda", dtype=torch.float64)
        for t in range(L):
            S.mul_(a[t][..., None, None]).addcmul_(k[t][..., :, None], v[t][..., None, :])
            torch.sum(S * q[t][..., :, None], -2, out=o[t])
        return o.permute(1, 2, 0, 3), S
    dO = by_token(s["dO"])
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S.mul_(a[t][..., None, None]).addcmul_(k[t][..., :, None], v[t][..., None, :])
        torch.sum(S * dO[t][..., None, :], -1, out=dq[t])
    dS = zero.clone() if s["dS"] is None else s["dS"].double()
    end = (S * dS).sum((-1, -2))
    for t in range(L - 1, -1, -1):
        dS.addcmul_(q[t][..., :, None], dO[t][..., None, :])
        torch.sum(dS * v[t][..., None, :], -1, out=dk[t])
        torch.sum(dS * k[t][..., :, None], -2, out=dv[t])
        dS.mul_(a[t][..., None, None])
    d = (q * dq).sum(-1) - (k * dk).sum(-1)
    dla = (end + d.flip(0).cumsum(0).flip(0)).permute(1, 2, 0)
    group = lambda t: t.permute(1, 2, 0, 3).reshape(B, Hk, H // Hk, L, Dk).sum(2)  # noqa: E731
    return {"dq": group(dq), "dk": group(dk), "dv": dv.permute(1, 2, 0, 3), "dS0": dS,
            "dlog_alpha": None if c["decay"] == "none" else dla if c["decay"] == "token" else dla.sum((0, 2))}


def exact(case, seed):
    c = case
    if c["op"] in ("fwd", "bwd"):
        # the loop over tokens moves every state once or more per token
        if c["L"] * (3e-5 + c["B"] * c["H"] * c["Dk"] * c["Dv"] * 8 * 6 / 2e12) * (3 if c["op"] == "bwd" else 1) > 15:
            return None
        return _exact_attention(case, seed)
    s = prepare(case, seed)
    if c["op"] == "step":
        rep = torch.arange(c["H"], device="cuda") // (c["H"] // c["Hk"])
        S = s["S"].double()
        if s["la"] is not None:
            a = s["la"].double().exp()
            S = S * (a.reshape(1, -1, 1, 1) if c["decay"] == "head" else a[..., None, None])
        S = S + s["k"].double()[:, rep][..., :, None] * s["v"].double()[..., None, :]
        return torch.matmul(s["q"].double()[:, rep][..., None, :], S)[..., 0, :], S
    x = s["x"].double()
    shape = (1, c["H"], 1, c["D"]) if c["per_head"] else (1, 1, 1, c["D"])
    w, b = s["w"].double().reshape(shape), s["b"].double().reshape(shape)
    if c["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        rstd = 1 / (var + EPS).sqrt()
        return (x - mean) * rstd * w + b, mean[..., 0], rstd[..., 0]
    mean, rstd, dy = s["mean"].double()[..., None], s["rstd"].double()[..., None], s["dy"].double()
    n = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.sum(-1, keepdim=True) / c["D"] - n * ((g * n).sum(-1, keepdim=True) / c["D"]))
    dw, db = (dy * n).sum((0, 2)), dy.sum((0, 2))
    return {"dx": dx, "dweight": dw if c["per_head"] else dw.sum(0), "dbias": db if c["per_head"] else db.sum(0)}
