"""The layer's operators together, as a model runs them: the norm with the residual's
addition, projections, the short convolution, the gated recurrence beside linear
attention, the norm per head, the way back, and the tokens after a prefill; against the
same chain in float64.

bf16 activations between the steps: every step rounds to 2^-9 of its values (2^-8 of
the smallest of a binade), a dozen of them carried through unit-scaled layers add up to
less than 2^-5 of a tensor's 2-norm."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import linattn_ref  # noqa: E402
import seqops_ref as ref  # noqa: E402
from seqops_ref import d  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def close(got, want, what, most=2.0 ** -5):
    err = float((d(got) - want).norm() / want.norm())
    assert err <= most, (what, err)


def mm(a, b):
    """[.., K] x [K, N], rounded to bf16 as a projection's output."""
    return (a.reshape(-1, a.shape[-1]) @ b).reshape(*a.shape[:-1], b.shape[-1])


def test_recurrent_block_trained_and_served():
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(21)
    B, L, D, W = 2, 333, 192, 4
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, res = r(B, L, D).to(BF).cuda(), (2 * r(B, L, D)).cuda()
    nw = (1 + 0.1 * r(D)).cuda()
    P = (r(D, 2 * D) / D ** 0.5).to(BF).cuda()
    cw, cb = (r(D, W) / 2).cuda(), (0.1 * r(D)).cuda()
    modes = dict(decay="logit", inputs="unit")
    dh, dres = r(B, L, D).to(BF).cuda(), (0.3 * r(B, L, D)).cuda()

    # forward: norm of the sum, one fused projection, convolution of its first half, gates from its second
    y, rstd, total = drl.dr_rmsnorm_fwd(x, nw, res)
    p = mm(y, P)
    u, cstate = drl.dr_short_conv_fwd(p[..., :D], cw, cb)
    h, last = drl.dr_gated_scan_fwd(u, p[..., D:], None, out_dtype=BF, **modes)
    # back
    gs = drl.dr_gated_scan_bwd(u, p[..., D:], None, h, dh, grad_dtype=BF, **modes)
    gc = drl.dr_short_conv_bwd(p[..., :D], cw, cb, None, gs["dx"])
    dp = torch.cat([gc["dx"], gs["dgate"]], -1)
    dy = mm(dp, P.t().contiguous())
    gn = drl.dr_rmsnorm_bwd(total, nw, rstd, dy, dres)

    X, R = d(x).requires_grad_(), d(res).requires_grad_()
    NW, PP, CW, CB = (d(t).requires_grad_() for t in (nw, P, cw, cb))
    s, wy, _ = ref.rms_forward(X, R, NW, 1e-5)
    wp = wy @ PP
    wu, wcs, _ = ref.conv_forward(wp[..., :D], CW, CB, None, True)
    wh, wlast = ref.scan_forward(wu, wp[..., D:], None, "logit", "unit")
    (wh * d(dh)).sum().backward(retain_graph=True)
    for got, want, what in ((y, wy, "y"), (u, wu, "u"), (cstate, wcs, "state"), (h, wh, "h"), (last, wlast, "last"),
                            (gc["dweight"], CW.grad, "dconv"), (gc["dbias"], CB.grad, "dbias"),
                            (gn["dweight"], NW.grad, "dnorm"), (gn["dx"], X.grad + d(dres), "dx")):
        close(got, want.detach(), what)
    assert torch.equal(total, x.float() + res)

    # served: 8-bit inputs of the projection for the next tokens, the states carried on
    y8, scale, _, _ = drl.dr_rmsnorm_fwd_e4m3(x, nw, res)
    back = y8.float() * scale.repeat_interleave(128, -1)[..., :D]
    close(back, wy.detach(), "8 bits", 2.0 ** -4)   # half a step of 3 bits
    with torch.no_grad():
        wc, wl = wcs.detach(), wlast.detach()
        for n in range(3):
            x1, r1 = r(B, D).to(BF).cuda(), (2 * r(B, D)).cuda()
            y1, _, _ = drl.dr_rmsnorm_fwd(x1, nw, r1)
            p1 = mm(y1, P)
            u1 = drl.dr_short_conv_step(cstate, p1[:, :D].contiguous(), cw, cb)
            h1 = drl.dr_gated_scan_step(last, u1, p1[:, D:].contiguous(), out_dtype=BF, **modes)
            _, wy1, _ = ref.rms_forward(d(x1), d(r1), d(nw), 1e-5)
            wp1 = (wy1 @ d(P))[:, None]
            wu1, wc, _ = ref.conv_forward(wp1[..., :D], d(cw), d(cb), wc, True)
            wh1, wl = ref.scan_forward(wu1, wp1[..., D:], wl, "logit", "unit")
            close(h1, wh1[:, 0], "next token")
            close(last, wl, "state")
            close(cstate, wc, "inputs")


def test_linear_attention_layer():
    """Convolutions of fused q, k, v rows as views, linear attention, RMS norm per head."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(22)
    B, L, H, D = 2, 200, 3, 64
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    qkv = r(B, L, 3 * H * D).to(BF).cuda()
    w = (r(3 * H * D, 4) / 2).cuda()
    la = -0.1 * torch.rand((H,), generator=gen).cuda()
    nw = (1 + 0.1 * r(H, D)).cuda()
    dy = r(B, L, H, D).to(BF).cuda().transpose(1, 2)
    c, _ = drl.dr_short_conv_fwd(qkv, w)
    q, k, v = (c[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).transpose(1, 2) for i in range(3))
    o, S = drl.dr_linear_attn_fwd(q, k, v, la, decay="head", out_dtype=BF)
    y, rstd, _ = drl.dr_rmsnorm_fwd(o, nw)
    gn = drl.dr_rmsnorm_bwd(o, nw, rstd, dy)
    ga = drl.dr_linear_attn_bwd(q, k, v, la, None, gn["dx"], decay="head", grad_dtype=BF)
    dc = torch.cat([ga[n].transpose(1, 2).flatten(-2) for n in ("dq", "dk", "dv")], -1)
    gc = drl.dr_short_conv_bwd(qkv, w, None, None, dc)

    Q = d(qkv)
    wc, _, _ = ref.conv_forward(Q, d(w), None, None, True)
    Wq, Wk, Wv = (wc[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).transpose(1, 2) for i in range(3))
    a = linattn_ref.gates(la, "head", B, H, L)
    wo, wS = linattn_ref.forward(Wq, Wk, Wv, a)
    _, wy, wr = ref.rms_forward(wo, None, d(nw)[None, :, None], 1e-5)
    wdx, wdw = ref.rms_backward(wo, d(nw)[None, :, None], wr, d(dy), None)
    dq, dk, dv, _, _ = linattn_ref.backward(Wq, Wk, Wv, a, None, wdx, None)
    wdc = torch.cat([t.transpose(1, 2).flatten(-2) for t in (dq, dk, dv)], -1)
    wg = ref.conv_backward(Q, d(w), None, None, wdc, None, True)
    for got, want, what in ((o, wo, "o"), (S, wS, "S"), (y, wy, "y"), (gn["dweight"], wdw.sum((0, 2)), "dnorm"),
                            (gc["dx"], wg["dx"], "dqkv"), (gc["dweight"], wg["dweight"], "dconv")):
        close(got, want, what)
