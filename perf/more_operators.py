"""The RMS norm with the residual's addition (forward, forward to 8 bits, backward), the short
causal convolution (forward, backward, one token) and the gated linear recurrence (forward,
backward, one token): the cases to measure, their inputs, their plain forms in elementary torch
operations, and their values in 64 bits.

    s = x + residual,  y = s rstd weight,  rstd = 1 / sqrt(mean(s^2) + eps)
    y_t = act(bias + sum_j w_j x_{t-W+1+j}),   act(z) = z or z sigmoid(z)
    h_t = a_t h_{t-1} + c_t x_t,   a = e^gate or sigmoid(gate),   c = 1, 1 - a or sqrt(1 - a^2)
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
BF16, F32, E4M3 = "bf16", "f32", "e4m3"


def _norm(name, op, B, H, L, D, per_head, dtype, res, out, token_major=False, block=128):
    return {"name": name, "op": op, "B": B, "H": H, "L": L, "D": D, "per_head": per_head, "dtype": dtype, "res": res,
            "out": out, "token_major": token_major, "block": block}


def _conv(name, op, B, L, C, W, dtype, out, act="silu", state=True, fused=False):
    return {"name": name, "op": op, "B": B, "L": L, "C": C, "W": W, "dtype": dtype, "out": out, "act": act,
            "state": state, "fused": fused}


def _scan(name, op, B, L, C, dtype, gate, out, decay, inputs, state=True):
    return {"name": name, "op": op, "B": B, "L": L, "C": C, "dtype": dtype, "gate": gate, "out": out, "decay": decay,
            "inputs": inputs, "state": state}


def listed():
    return [
        # a block's norm over the model width, the residual stream in bf16: prefill or training
        _norm("norm residual", "norm_fwd", 1, 1, 8191, 2048, False, BF16, BF16, BF16),
        # a large batch's norm in front of 8-bit products: a scale for each 128 values, the stream in fp32
        _norm("norm 8 bits", "norm_fwd", 1, 1, 16384, 4096, False, BF16, F32, E4M3),
        # one conversation's next token, a scale for the row; latency counts
        _norm("norm next token", "norm_fwd", 1, 1, 1, 2048, False, BF16, BF16, E4M3, block=0),
        # the backward of the first, with the stream's own gradient
        _norm("norm bwd", "norm_bwd", 1, 1, 8191, 2048, False, BF16, BF16, BF16),
        # the convolution of the long prefill's values, a slice of a fused projection
        _conv("conv long", "conv_fwd", 2, 16384, 2048, 4, BF16, BF16, fused=True),
        # training at that shape
        _conv("conv bwd long", "conv_bwd", 2, 16384, 2048, 4, BF16, BF16),
        # the decode batch's next token
        _conv("conv step", "conv_step", 256, 1, 2048, 4, BF16, BF16),
        # a recurrent layer on the long prefill, gates as its projection leaves them
        _scan("scan long", "scan_fwd", 2, 16384, 2048, BF16, BF16, BF16, "logit", "unit"),
        # one long sequence of few channels in fp32
        _scan("scan narrow", "scan_fwd", 1, 65536, 200, F32, F32, F32, "log", "plain"),
        # training at the long shape
        _scan("scan bwd long", "scan_bwd", 2, 16384, 2048, BF16, BF16, BF16, "logit", "blend"),
        # training on a small batch of odd length and width, gradients kept in 32 bits
        _scan("scan bwd ragged", "scan_bwd", 3, 1111, 1001, BF16, F32, F32, "log", "plain"),
        # the decode batch's next token
        _scan("scan step", "scan_step", 256, 1, 2048, BF16, BF16, BF16, "logit", "unit"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, hi):
    """Channels: whole multiples of 8 as a rule, others too."""
    C = _log_int(rng, 16, hi)
    return C if rng.random() < 0.3 else max(8, C // 8 * 8)


MOST = 2 * 16384 * 2048   # values of the largest listed tensors


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd",
                     "scan_bwd", "scan_bwd", "scan_step"))
    dtype = rng.choice((BF16, BF16, BF16, F32))
    out = F32 if dtype == F32 else rng.choice((BF16, BF16, F32))
    if op.startswith("norm"):
        out = E4M3 if op == "norm_fwd" and rng.random() < 0.5 else out
        res = rng.choice((dtype, F32, "none"))
        if rng.random() < 0.3:
            D, H, heads = rng.choice((64, 128, 8 * rng.randint(1, 32))), rng.choice((1, 2, 8, 16)), True
            L = _log_int(rng, 1, min(16384, MOST // (2 * H * D)))
            B = _log_int(rng, 1, max(1, min(64, MOST // (2 * H * L * D))))
        else:
            D, B, H, heads = _width(rng, 16384), 1, 1, False
            L = _log_int(rng, 1, MOST // (2 * max(D, 128)))
        if out == E4M3:
            D = max(8, D // 8 * 8)
        case = _norm("", op, B, H, L, D, heads, dtype, res, out, token_major=heads and rng.random() < 0.5,
                     block=rng.choice((128, 128, 0)))
    else:
        C = _width(rng, 8192)
        most = MOST // (1 if dtype == BF16 else 2)
        if op.endswith("step"):
            B, L = _log_int(rng, 1, 1024), 1
        else:
            L = _log_int(rng, 1, 65536)
            B = _log_int(rng, 1, max(1, min(256, most // (C * L))))
            L = max(1, min(L, most // (B * C)))
        if op.startswith("conv"):
            case = _conv("", op, B, L, C, rng.choice((2, 3, 4, 4, 4, 5, 8)), dtype, out, rng.choice(("silu", "silu", "none")),
                         state=rng.random() < 0.7 or op == "conv_step", fused=rng.random() < 0.3 and op == "conv_fwd")
        else:
            case = _scan("", op, B, L, C, dtype, rng.choice((dtype, F32)), out, rng.choice(("log", "logit")),
                         rng.choice(("plain", "blend", "unit")), state=rng.random() < 0.7 or op == "scan_step")
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _type(name):
    return {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}[name]


def _gates(gen, shape, c):
    """Decays of 1 to 1000 tokens' memory: logs in [-0.1, -0.001], or logits around 3."""
    if c["decay"] == "log":
        g = -(0.001 + 0.099 * torch.rand(shape, device="cuda", generator=gen))
    else:
        g = 3 + 1.5 * torch.randn(shape, device="cuda", generator=gen)
    return g.to(_type(c["gate"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": dict(case)}

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    if c["op"].startswith("norm"):
        B, H, L, D = (c[n] for n in ("B", "H", "L", "D"))

        def rows(dtype):
            x = normal(B, L, H, D).to(_type(dtype)).transpose(1, 2) if c["token_major"] else normal(B, H, L, D).to(_type(dtype))
            return x if c["per_head"] else x.reshape(L, D)

        s["x"] = rows(c["dtype"])
        s["w"] = 1 + 0.1 * normal(*((H, D) if c["per_head"] else (D,)))
        if c["op"] == "norm_fwd":
            s["r"] = None if c["res"] == "none" else 3 * rows(c["res"])
        else:
            s["dy"] = rows(c["dtype"])
            s["ds"] = None if c["res"] == "none" else rows(c["res"])
            s["rstd"] = (s["x"].double().square().mean(-1) + EPS).rsqrt().float().contiguous()
        return s
    B, L, C, t = c["B"], c["L"], c["C"], _type(c["dtype"])
    if c["op"].startswith("conv"):
        W = c["W"]
        x = normal(B, L, C).to(t)
        if c["fused"]:
            x = torch.cat([torch.empty_like(x), x], -1)[..., C:]   # the second half of a projection's rows
        s["x"] = x[:, 0] if c["op"] == "conv_step" else x
        s["w"], s["b"] = normal(C, W) / math.sqrt(W), 0.1 * normal(C)
        s["state"] = normal(B, W - 1, C).to(t) if c["state"] else None
        if c["op"] == "conv_bwd":
            s["dy"] = normal(B, L, C).to(t)
            s["dstate"] = normal(B, W - 1, C) if c["state"] else None
        return s
    s["x"], s["g"] = normal(B, L, C).to(t), _gates(gen, (B, L, C), c)
    s["h0"] = normal(B, C) if c["state"] else None
    if c["op"] == "scan_step":
        s["x"], s["g"] = s["x"][:, 0].contiguous(), s["g"][:, 0].contiguous()
    if c["op"] == "scan_bwd":
        s["h"] = _plain_scan_fwd(s)[0]
        s["dh"] = normal(B, L, C).to(t)
        s["dlast"] = normal(B, C) if c["state"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _plain_norm_fwd(s):
    c = s["case"]
    x = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    total = None if s["r"] is None else x.to(s["r"].dtype)
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = x * rstd * (s["w"][None, :, None] if c["per_head"] else s["w"])
    if c["out"] != E4M3:
        return y.to(_type(c["out"])), rstd[..., 0], total
    n = c["block"] or c["D"]
    blocks = torch.nn.functional.pad(y, (0, -c["D"] % n)).unflatten(-1, (-1, n))
    scale = (blocks.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
    codes = (blocks / scale[..., None]).flatten(-2)[..., :c["D"]].contiguous().to(torch.float8_e4m3fn)
    return codes, scale, rstd[..., 0], total


def _plain_norm_bwd(s):
    c = s["case"]
    dy, r = s["dy"].float(), s["rstd"][..., None]
    n = s["x"].float() * r
    t = dy * (s["w"][None, :, None] if c["per_head"] else s["w"])
    dx = r * (t - n * (t * n).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"dx": dx.to(_type(c["out"])), "dweight": (dy * n).sum((0, 2) if c["per_head"] else 0)}


def _past(s):
    """The rows of x behind those of the state (zeros without one), in fp32."""
    B, L, C = s["x"].shape
    first = s["x"].new_zeros(B, s["case"]["W"] - 1, C) if s["state"] is None else s["state"]
    return torch.cat([first, s["x"]], 1)


def _taps(x, w, L):
    return sum(x[:, j:j + L] * w[:, j] for j in range(w.shape[1]))


def _plain_conv_fwd(s):
    c, L = s["case"], s["x"].shape[1]
    past = _past(s)
    z = _taps(past.float(), s["w"], L) + s["b"]
    y = z * torch.sigmoid(z) if c["act"] == "silu" else z
    return y.to(_type(c["out"])), past[:, L:].contiguous()


def _plain_conv_bwd(s):
    c, (B, L, C) = s["case"], s["x"].shape
    W, past, dz = c["W"], _past(s).float(), s["dy"].float()
    if c["act"] == "silu":
        z = _taps(past, s["w"], L) + s["b"]
        p = torch.sigmoid(z)
        dz = dz * p * (1 + z * (1 - p))
    d = torch.zeros_like(past)
    for j in range(W):
        d[:, j:j + L] += s["w"][:, j] * dz
    if s["dstate"] is not None:
        d[:, L:] += s["dstate"]
    dw = torch.stack([(dz * past[:, j:j + L]).sum((0, 1)) for j in range(W)], -1)
    return {"dx": d[:, W - 1:].to(_type(c["out"])), "dweight": dw, "dbias": dz.sum((0, 1)),
            "dstate": d[:, :W - 1].contiguous()}


def _plain_conv_step(s):
    c = s["case"]
    past = torch.cat([s["state"], s["x"][:, None]], 1)
    z = (past.float() * s["w"].t()).sum(1) + s["b"]
    s["state"].copy_(past[:, 1:])
    return (z * torch.sigmoid(z) if c["act"] == "silu" else z).to(_type(c["out"])), s["state"]


def _factors(s):
    """a, 1 - a and the input's factor c, in fp32."""
    c, g = s["case"], s["g"].float()
    if c["decay"] == "log":
        a, rest = g.exp(), -torch.expm1(g)
    else:
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    return a, rest, {"plain": None, "blend": rest, "unit": (rest * (1 + a)).sqrt()}[c["inputs"]]


def _doubling(a, b):
    """b_t + a_t (b_{t-1} + a_{t-1} (...)) along the tokens, spans doubled log2(L) times."""
    n = 1
    while n < b.shape[1]:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _plain_scan_fwd(s):
    a, _, f = _factors(s)
    b = s["x"].float() if f is None else f * s["x"].float()
    if s["h0"] is not None:
        b = torch.cat([b[:, :1] + a[:, :1] * s["h0"][:, None], b[:, 1:]], 1)
    h = _doubling(a, b)
    return h.to(_type(s["case"]["out"])), h[:, -1].contiguous()


def _plain_scan_bwd(s):
    c = s["case"]
    a, rest, f = _factors(s)
    x, dh = s["x"].float(), s["dh"].float()
    if s["dlast"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dlast"][:, None]], 1)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)   # a_{t+1}
    d = _doubling(after.flip(1), dh.flip(1)).flip(1)
    first = torch.zeros_like(x[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([first, s["h"][:, :-1].float()], 1)        # h_{t-1}
    if c["inputs"] == "blend":
        before = before - x
    elif c["inputs"] == "unit":
        before = before - a / f * x
    dg = d * before * (a if c["decay"] == "log" else a * rest)
    to = _type(c["out"])
    return {"dx": (d if f is None else f * d).to(to), "dgate": dg.to(to), "dh0": a[:, 0] * d[:, 0]}


def _plain_scan_step(s):
    a, _, f = _factors(s)
    s["h0"].mul_(a).add_(s["x"].float() if f is None else f * s["x"].float())
    return s["h0"].to(_type(s["case"]["out"])), s["h0"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "conv_fwd": _plain_conv_fwd,
                "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step, "scan_fwd": _plain_scan_fwd,
                "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step}[op](s)
    import delta_rule_linear_amd as drl
    to = _type(c["out"])
    if op == "norm_fwd" and c["out"] == E4M3:
        return drl.dr_rmsnorm_fwd_e4m3(s["x"], s["w"], s["r"], eps=EPS, block=c["block"])
    if op == "norm_fwd":
        return drl.dr_rmsnorm_fwd(s["x"], s["w"], s["r"], eps=EPS, out_dtype=to)
    if op == "norm_bwd":
        return drl.dr_rmsnorm_bwd(s["x"], s["w"], s["rstd"], s["dy"], s["ds"], grad_dtype=to)
    if op == "conv_fwd":
        return drl.dr_short_conv_fwd(s["x"], s["w"], s["b"], s["state"], activation=c["act"], out_dtype=to)
    if op == "conv_bwd":
        return drl.dr_short_conv_bwd(s["x"], s["w"], s["b"], s["state"], s["dy"], s["dstate"], activation=c["act"],
                                     grad_dtype=to)
    if op == "conv_step":
        return drl.dr_short_conv_step(s["state"], s["x"], s["w"], s["b"], activation=c["act"], out_dtype=to), s["state"]
    mode = {"decay": c["decay"], "inputs": c["inputs"]}
    if op == "scan_fwd":
        return drl.dr_gated_scan_fwd(s["x"], s["g"], s["h0"], out_dtype=to, **mode)
    if op == "scan_bwd":
        return drl.dr_gated_scan_bwd(s["x"], s["g"], s["h0"], s["h"], s["dh"], s["dlast"], grad_dtype=to, **mode)
    return drl.dr_gated_scan_step(s["h0"], s["x"], s["g"], out_dtype=to, **mode), s["h0"]


def work(case):
    c = case
    size = {BF16: 2, F32: 4, E4M3: 1, "none": 0}
    i, o = size[c["dtype"]], size[c["out"]]
    if c["op"].startswith("norm"):
        rows, D, r = c["B"] * c["H"] * c["L"], c["D"], size[c["res"]]
        w = 4 * D * (c["H"] if c["per_head"] else 1)
        if c["op"] == "norm_bwd":
            return {"bytes": rows * (D * (2 * i + r + o) + 4) + 2 * w, "flops": 10 * rows * D}
        scales = 4 * rows * (-(-D // c["block"]) if c["block"] else 1) if c["out"] == E4M3 else 0
        return {"bytes": rows * (D * (i + 2 * r + o) + 4) + w + scales, "flops": 6 * rows * D}
    n, BC = c["B"] * c["L"] * c["C"], c["B"] * c["C"]
    if c["op"].startswith("conv"):
        W = c["W"]
        state, w = BC * (W - 1) * i * (2 if c["state"] else 1), 4 * c["C"] * (W + 1)
        if c["op"] == "conv_bwd":
            state = BC * (W - 1) * (i + 8 if c["state"] else 4)
            return {"bytes": n * (2 * i + o) + state + 2 * w, "flops": n * (6 * W + 12)}
        return {"bytes": n * (i + o) + state + w, "flops": n * (2 * W + 5)}
    g, state = size[c["gate"]], 4 * BC * (2 if c["state"] else 1)
    if c["op"] == "scan_bwd":
        # x is needed where its factor depends on the gate
        ins = g + size[c["out"]] + i + (0 if c["inputs"] == "plain" else i)
        return {"bytes": n * (ins + 2 * o) + state + 4 * BC, "flops": 14 * n}
    return {"bytes": n * (i + g + o) + state, "flops": 8 * n}


# ---------------------------------------------------------------- in 64 bits

def _e4m3(v):
    """v to the nearest value with 3 bits behind the leading one, ties to even, steps of 2^-9 at least."""
    step = torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4)
    return (v / step).round() * step


def _exact_norm(c, s):
    x = s["x"].double()
    w = s["w"].double()
    if c["per_head"]:
        w = w.reshape(1, c["H"], 1, c["D"])
    if c["op"] == "norm_bwd":
        rstd, dy = s["rstd"].double().unsqueeze(-1), s["dy"].double()
        n, t = x * rstd, dy * w
        dx = rstd * t - rstd * n * ((t * n).sum(-1, keepdim=True) / c["D"])
        if s["ds"] is not None:
            dx += s["ds"].double()
        dw = dy * n
        return {"dx": dx, "dweight": dw.sum(2).sum(0) if c["per_head"] else dw.sum(0)}
    if s["r"] is not None:
        x = x + s["r"].double()
    rstd = 1 / torch.sqrt((x * x).sum(-1) / c["D"] + EPS)
    y = x * rstd.unsqueeze(-1) * w
    total = None if s["r"] is None else x
    if c["out"] != E4M3:
        return y, rstd, total
    n = c["block"] or c["D"]
    scales = [y[..., i:i + n].abs().amax(-1) / E4M3_MAX for i in range(0, c["D"], n)]
    codes = [_e4m3(y[..., k * n:(k + 1) * n] / a.unsqueeze(-1)) for k, a in enumerate(scales)]
    return torch.cat(codes, -1), torch.stack(scales, -1), rstd, total


def _exact_conv(c, s):
    W, w, b = c["W"], s["w"].double(), s["b"].double()
    x = s["x"].double()
    x = x.unsqueeze(1) if c["op"] == "conv_step" else x
    B, L, C = x.shape
    past = torch.zeros(B, L + W - 1, C, dtype=torch.float64, device=x.device)
    past[:, W - 1:] = x
    if s["state"] is not None:
        past[:, :W - 1] = s["state"].double()
    rows = past.unfold(1, W, 1)                    # [B, L, C, W]
    z = torch.empty_like(x)
    for i in range(0, L, 4096):                    # the products of 4096 tokens at a time
        z[:, i:i + 4096] = (rows[:, i:i + 4096] * w).sum(-1) + b
    e = torch.exp(-z) if c["act"] == "silu" else torch.zeros_like(z)
    if c["op"] != "conv_bwd":
        y, last = z / (1 + e), past[:, L:]
        return (y[:, 0] if c["op"] == "conv_step" else y), last
    dz = s["dy"].double()
    if c["act"] == "silu":
        dz = dz * (1 / (1 + e) + z * e / (1 + e) ** 2)
    wide = torch.zeros(B, L + 2 * (W - 1), C, dtype=torch.float64, device=x.device)
    wide[:, W - 1:W - 1 + L] = dz                  # past row i enters the outputs i - W + 1 .. i
    d = torch.zeros_like(past)
    dw = torch.empty(C, W, dtype=torch.float64, device=x.device)
    for j in range(W):
        d += w[:, W - 1 - j] * wide[:, j:j + L + W - 1]
        dw[:, j] = torch.einsum("blc,blc->c", dz, past[:, j:j + L])
    if s["dstate"] is not None:
        d[:, L:] += s["dstate"].double()
    return {"dx": d[:, W - 1:], "dweight": dw, "dbias": dz.sum(1).sum(0), "dstate": d[:, :W - 1]}


def _exact_scan(c, s):
    g = s["g"].double()
    x = s["x"].double()
    if c["op"] == "scan_step":
        g, x = g.unsqueeze(1), x.unsqueeze(1)
    B, L, C = x.shape
    a = torch.exp(g) if c["decay"] == "log" else 1 / (1 + torch.exp(-g))
    rest = 1 - a                                   # 53 bits hold it to 2^-43 at the weakest decay
    f = {"plain": torch.ones_like(a), "blend": rest, "unit": torch.sqrt(rest * (1 + a))}[c["inputs"]]
    by_token = lambda t: t.transpose(0, 1).contiguous()  # noqa: E731
    at = by_token(a)
    h0 = torch.zeros(B, C, dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    if c["op"] != "scan_bwd":
        h, u = h0, by_token(f * x)
        for t in range(L):
            torch.addcmul(u[t], at[t], h, out=u[t])
            h = u[t]
        out = u.transpose(0, 1)
        return (out[:, 0] if c["op"] == "scan_step" else out), h
    d = by_token(s["dh"].double())
    if s["dlast"] is not None:
        d[L - 1] += s["dlast"].double()
    for t in range(L - 2, -1, -1):
        torch.addcmul(d[t], at[t + 1], d[t + 1], out=d[t])
    d = d.transpose(0, 1)
    before = torch.empty_like(x)
    before[:, 0] = h0
    before[:, 1:] = s["h"][:, :-1].double()
    da = {"plain": 0.0, "blend": -x, "unit": -a / f * x}[c["inputs"]] + before
    return {"dx": f * d, "dgate": da * d * (a if c["decay"] == "log" else a * rest), "dh0": a[:, 0] * d[:, 0]}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("norm"):
        return _exact_norm(c, s)
    if c["op"].startswith("conv"):
        return _exact_conv(c, s)
    if c["L"] * (1e-5 + c["B"] * c["C"] * 32 / 2e12) > 15:   # the loop over the tokens
        return None
    return _exact_scan(c, s)
