"""The host side of linear attention and layer norm without a GPU: bad
arguments are refused before any device work (the fake pointers are never
touched), and the float64 oracle's gradients agree with autograd and with
differences."""
import ctypes

import pytest

import delta_rule_linear_amd as drl

torch = pytest.importorskip("torch")
import linattn_ref as ref  # noqa: E402

FAKE = 0x7f0000000000


def F(i):
    """Fake tensor addresses 64 GiB apart."""
    return FAKE + (i << 36)


def desc(**kw):
    base = dict(B=2, H=6, Hk=3, L=5000, Dk=64, Dv=128, in_dtype=drl.DR_BF16, out_dtype=drl.DR_F32, decay="token")
    base.update(kw)
    return drl.linattn_desc(**base)


NAMES = ("q", "k", "v", "la", "S0", "o", "Sf", "ws")


def fwd(d, wbytes=1 << 40, **kw):
    p = {n: F(i) for i, n in enumerate(NAMES)}
    p.update(kw)
    return drl.lib().dr_linear_attn_fwd(ctypes.byref(d) if d is not None else None, *(p[n] for n in NAMES), wbytes, None)


BNAMES = ("q", "k", "v", "la", "S0", "dO", "dS", "dq", "dk", "dv", "dla", "dS0", "ws")


def bwd(d, wbytes=1 << 40, **kw):
    p = {n: F(i) for i, n in enumerate(BNAMES)}
    p.update(kw)
    return drl.lib().dr_linear_attn_bwd(ctypes.byref(d) if d is not None else None, *(p[n] for n in BNAMES), wbytes,
                                        None)


@pytest.mark.parametrize("kw,code", [
    (dict(Dk=0), drl.DR_ERR_UNSUPPORTED),
    (dict(Dk=4), drl.DR_ERR_UNSUPPORTED),
    (dict(Dk=100), drl.DR_ERR_UNSUPPORTED),
    (dict(Dv=136), drl.DR_ERR_UNSUPPORTED),
    (dict(Hk=4), drl.DR_ERR_UNSUPPORTED),
    (dict(Hk=0), drl.DR_ERR_SHAPE),
    (dict(Hk=-3), drl.DR_ERR_SHAPE),
    (dict(L=-1), drl.DR_ERR_SHAPE),
    (dict(B=-1), drl.DR_ERR_SHAPE),
    (dict(L=2 ** 31 - 1), drl.DR_ERR_UNSUPPORTED),
    (dict(B=2 ** 30, H=6), drl.DR_ERR_UNSUPPORTED),
    (dict(in_dtype=2), drl.DR_ERR_UNSUPPORTED),
    (dict(out_dtype=-1), drl.DR_ERR_UNSUPPORTED),
])
def test_bad_descriptors(kw, code):
    for call in (fwd, bwd):
        assert call(desc(**kw)) == code
        assert drl.dr_last_error()
    assert drl.dr_linear_attn_fwd_workspace_bytes(desc(**kw)) == 0
    assert drl.dr_linear_attn_bwd_workspace_bytes(desc(**kw)) == 0


def test_unknown_decay_and_null():
    d = desc()
    d.decay = 3
    assert fwd(d) == bwd(d) == drl.DR_ERR_UNSUPPORTED
    assert fwd(None) == bwd(None) == drl.DR_ERR_NULL
    for n in ("q", "k", "v", "o", "la"):
        assert fwd(desc(), **{n: None}) == drl.DR_ERR_NULL
    for n in ("q", "k", "v", "dO", "dq", "dk", "dv", "la", "dla"):
        assert bwd(desc(), **{n: None}) == drl.DR_ERR_NULL
    assert fwd(desc(decay="none")) == bwd(desc(decay="none")) == drl.DR_ERR_NULL
    assert bwd(desc(decay="none"), la=None) == drl.DR_ERR_NULL


def test_alignment_and_strides():
    for n in ("q", "k", "v", "la", "S0", "o", "Sf", "ws"):
        assert fwd(desc(), **{n: F(20) + 8}) == drl.DR_ERR_ALIGN, n
    for n in BNAMES:
        assert bwd(desc(), **{n: F(20) + 4}) == drl.DR_ERR_ALIGN, n
    for f in ("q", "k", "v", "o"):
        d = desc()
        getattr(d, f).t = 66
        assert fwd(d) == drl.DR_ERR_ALIGN
        d = desc()
        getattr(d, f).h = -64
        assert fwd(d) == drl.DR_ERR_SHAPE
    # rows of an output that share memory
    for f, call in (("o", fwd), ("dq", bwd), ("dk", bwd), ("dv", bwd)):
        d = desc()
        getattr(d, f).t = 32
        assert call(d) == drl.DR_ERR_UNSUPPORTED and "overlap" in drl.dr_last_error()
        d = desc()
        getattr(d, f).b = 0
        assert call(d) == drl.DR_ERR_UNSUPPORTED
    # a dimension of one has no stride
    d = desc(B=1)
    d.q.b = d.o.b = 3
    assert fwd(d, ws=None) == drl.DR_ERR_WORKSPACE


def test_overlaps():
    assert fwd(desc(), o=F(0)) == drl.DR_ERR_UNSUPPORTED
    assert fwd(desc(), Sf=F(5) + 16) == drl.DR_ERR_UNSUPPORTED
    assert fwd(desc(), Sf=F(4) + 16) == drl.DR_ERR_UNSUPPORTED     # S_final inside S0, not S0 itself
    assert fwd(desc(), Sf=F(4), ws=None) == drl.DR_ERR_WORKSPACE   # in place: validation goes on
    assert fwd(desc(), ws=F(5) + 256) == drl.DR_ERR_UNSUPPORTED
    assert bwd(desc(), dq=F(1)) == drl.DR_ERR_UNSUPPORTED
    assert bwd(desc(), dk=F(7) + 16) == drl.DR_ERR_UNSUPPORTED
    assert bwd(desc(), dS0=F(4)) == drl.DR_ERR_UNSUPPORTED


def test_workspaces():
    d = desc()
    need = drl.dr_linear_attn_fwd_workspace_bytes(d)
    assert need > 0 and need % 256 == 0
    assert fwd(d, ws=None) == fwd(d, wbytes=need - 1) == drl.DR_ERR_WORKSPACE
    # many sequences need no segments
    assert drl.dr_linear_attn_fwd_workspace_bytes(desc(B=128)) == 0
    need = drl.dr_linear_attn_bwd_workspace_bytes(d)
    assert bwd(d, wbytes=need - 1) == drl.DR_ERR_WORKSPACE
    # shared heads: fp32 gradients of q and k for every state head
    own = drl.dr_linear_attn_bwd_workspace_bytes(desc(Hk=6))
    assert need - own == 2 * 2 * 6 * 5000 * 64 * 4
    for e in (desc(L=0), desc(B=0), desc(H=0)):
        assert drl.dr_linear_attn_fwd_workspace_bytes(e) == drl.dr_linear_attn_bwd_workspace_bytes(e) == 0


def test_step_refusals():
    S = drl.LinAttnStepDesc
    ok = dict(N=4, H=6, Hk=3, Dk=64, Dv=128, in_dtype=1, out_dtype=0, decay=2)

    def call(kw=None, **ptr):
        p = {n: F(i) for i, n in enumerate(("q", "k", "v", "la", "S", "o"))}
        p.update(ptr)
        return drl.lib().dr_linear_attn_step(ctypes.byref(S(**{**ok, **(kw or {})})), *p.values(), None)

    for kw in (dict(Dk=12), dict(Dv=256), dict(Hk=5), dict(decay=9), dict(in_dtype=7)):
        assert call(kw) == drl.DR_ERR_UNSUPPORTED
    assert call(dict(N=-1)) == call(dict(Hk=0)) == drl.DR_ERR_SHAPE
    for n in ("q", "k", "v", "la", "S", "o"):
        assert call(**{n: None}) == drl.DR_ERR_NULL
        assert call(**{n: F(9) + 8}) == drl.DR_ERR_ALIGN
    assert call(dict(decay=0)) == drl.DR_ERR_NULL
    assert call(o=F(4)) == call(S=F(2)) == drl.DR_ERR_UNSUPPORTED
    assert call(dict(N=0)) == drl.DR_OK
    assert drl.lib().dr_linear_attn_step(None, *[F(i) for i in range(6)], None) == drl.DR_ERR_NULL


def ln(**kw):
    base = dict(B=2, H=4, L=100, D=128, per_head=1, x_dtype=1, y_dtype=0, dy_dtype=1, eps=1e-5)
    base.update(kw)
    B, H, L, D = (base[n] for n in ("B", "H", "L", "D"))
    s = drl.Strides(H * L * D, L * D, D)
    return drl.LayerNormDesc(**base, x=s, y=s, dy=s)


def lnf(d, **kw):
    p = {n: F(i) for i, n in enumerate(("x", "w", "b", "y", "mean", "rstd"))}
    p.update(kw)
    return drl.lib().dr_layernorm_fwd(ctypes.byref(d), *p.values(), None)


def lnb(d, wbytes=1 << 40, **kw):
    p = {n: F(i) for i, n in enumerate(("x", "w", "mean", "rstd", "dy", "dx", "dw", "db", "ws"))}
    p.update(kw)
    return drl.lib().dr_layernorm_bwd(ctypes.byref(d), *p.values(), wbytes, None)


def test_layernorm_refusals():
    for kw in (dict(D=0), dict(D=16385), dict(per_head=2), dict(x_dtype=5), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(B=2 ** 16, H=1, L=2 ** 16)):
        assert lnf(ln(**kw)) == lnb(ln(**kw)) == drl.DR_ERR_UNSUPPORTED, kw
        assert drl.dr_layernorm_bwd_workspace_bytes(ln(**kw)) == 0
    assert lnf(ln(L=-1)) == lnb(ln(L=-1)) == drl.DR_ERR_SHAPE
    for n in ("x", "y"):
        assert lnf(ln(), **{n: None}) == drl.DR_ERR_NULL
    for n in ("x", "mean", "rstd", "dy", "dx"):
        assert lnb(ln(), **{n: None}) == drl.DR_ERR_NULL
    for n in ("x", "w", "b", "y", "mean", "rstd"):
        assert lnf(ln(), **{n: F(9) + 4}) == drl.DR_ERR_ALIGN
    assert lnf(ln(), y=F(0)) == lnf(ln(), mean=F(3)) == drl.DR_ERR_UNSUPPORTED
    assert lnb(ln(), dx=F(4)) == lnb(ln(), dw=F(7)) == drl.DR_ERR_UNSUPPORTED
    d = ln()
    d.y.t = 64
    assert lnf(d) == lnb(d) == drl.DR_ERR_UNSUPPORTED
    d = ln()
    d.x.h = -128
    assert lnf(d) == drl.DR_ERR_SHAPE
    need = drl.dr_layernorm_bwd_workspace_bytes(ln())
    assert need > 0
    assert lnb(ln(), wbytes=need - 1) == lnb(ln(), ws=None) == drl.DR_ERR_WORKSPACE
    assert lnf(ln(L=0)) == drl.DR_OK


def test_strides_past_any_memory():
    """A last row more than 2^48 elements behind the first is refused, also
    where the product of stride and rows passes 64 bits."""
    for f in ("q", "k", "v", "o"):
        d = desc(B=2 ** 12, H=3)
        getattr(d, f).b = 2 ** 40
        assert fwd(d) == drl.DR_ERR_SHAPE and "too large" in drl.dr_last_error()
    d = ln(B=2 ** 20, H=1, L=2)
    d.x.b = 2 ** 47
    assert lnf(d) == lnb(d) == drl.DR_ERR_SHAPE


def test_binding_needs_device_tensors():
    x = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        drl.dr_linear_attn_fwd(x, x, x, decay="none")
    with pytest.raises(ValueError, match="device tensor"):
        drl.dr_layernorm_fwd(x)
    with pytest.raises(ValueError, match="channels"):
        drl.dr_linear_attn_fwd(x[0], x[0], x[0], decay="none")


@pytest.mark.parametrize("decay", ["none", "head", "token"])
def test_oracle_gradients(decay):
    """The oracle's formulas against autograd through its forward, in float64."""
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, H, Hk, L, Dk, Dv = 2, 4, 2, 9, 3, 5
    q, k, v, S0, dO, dS = r(B, Hk, L, Dk), r(B, Hk, L, Dk), r(B, H, L, Dv), r(B, H, Dk, Dv), r(B, H, L, Dv), r(B, H, Dk, Dv)
    la = None if decay == "none" else -torch.rand((H,) if decay == "head" else (B, H, L), generator=gen,
                                                 dtype=torch.float64)
    want, size = ref.reference(q, k, v, la, S0, decay, dO, dS)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, S0)] + ([] if la is None else [la.clone().requires_grad_()])
    o, S = ref.forward(ref.heads(leaves[0], H), ref.heads(leaves[1], H), leaves[2],
                       ref.gates(None, "none", B, H, L) if la is None else
                       (leaves[4].exp()[None, :, None].expand(B, H, L) if decay == "head" else leaves[4].exp()),
                       leaves[3])
    grads = torch.autograd.grad((o * dO).sum() + (S * dS).sum(), leaves)
    for name, g in zip(("dq", "dk", "dv", "dS0", "dlog_alpha"), grads):
        assert torch.allclose(g, want[name], rtol=1e-10, atol=1e-10), name
        assert (size[name] >= want[name].abs() - 1e-9).all()


def test_oracle_norm_gradients():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    for per_head in (False, True):
        x, dy = r(2, 3, 4, 6), r(2, 3, 4, 6)
        w, b = (r(3, 6), r(3, 6)) if per_head else (r(6), r(6))
        leaves = [t.clone().requires_grad_() for t in (x, w, b)]
        y, mean, rstd = ref.norm_forward(*leaves, 1e-5)
        want = torch.autograd.grad((y * dy).sum(), leaves)
        got = ref.norm_backward(x, w, mean.detach(), rstd.detach(), dy, per_head)
        for a, c in zip(got, want):
            assert torch.allclose(a, c, rtol=1e-9, atol=1e-9)
