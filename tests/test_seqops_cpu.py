"""The host side of the RMS norm, the short convolution and the gated recurrence
without a GPU: bad arguments are refused before any device work (the fake pointers
are never touched), and the float64 oracle's gradients agree with autograd."""
import ctypes

import pytest

import delta_rule_linear_amd as drl

torch = pytest.importorskip("torch")
import seqops_ref as ref  # noqa: E402

FAKE = 0x7f0000000000
BIG = 1 << 40


def F(i):
    """Fake tensor addresses 64 GiB apart."""
    return FAKE + (i << 36)


def call(name, d, names, given, wbytes=None):
    p = {n: F(i) for i, n in enumerate(names)}
    p.update(given)
    tail = [] if wbytes is None else [wbytes]
    return getattr(drl.lib(), name)(ctypes.byref(d) if d is not None else None, *(p[n] for n in names), *tail, None)


def S(b, h, t):
    return drl.Strides(b, h, t)


# ---------------------------------------------------------------- RMS norm

def rn(**kw):
    base = dict(B=2, H=3, L=50, D=200, per_head=1, x_dtype=drl.DR_BF16, res_dtype=drl.DR_F32, y_dtype=drl.DR_BF16,
                dy_dtype=drl.DR_F32, eps=1e-5, block=128)
    base.update(kw)
    H, L, D = base["H"], base["L"], base["D"]
    dense = S(H * L * D, L * D, D)
    return drl.RMSNormDesc(*base.values(), *(dense,) * 5)


RF = ("x", "residual", "weight", "y", "total", "rstd")
RE = ("x", "residual", "weight", "y", "scale", "total", "rstd")
RB = ("x", "weight", "rstd", "dy", "ds", "dx", "dweight", "ws")


def rf(d, **kw):
    return call("dr_rmsnorm_fwd", d, RF, kw)


def re_(d, **kw):
    return call("dr_rmsnorm_fwd_e4m3", d, RE, kw)


def rb(d, wbytes=BIG, **kw):
    return call("dr_rmsnorm_bwd", d, RB, kw, wbytes)


@pytest.mark.parametrize("kw,code", [
    (dict(D=0), drl.DR_ERR_UNSUPPORTED), (dict(D=16385), drl.DR_ERR_UNSUPPORTED), (dict(L=-1), drl.DR_ERR_SHAPE),
    (dict(per_head=2), drl.DR_ERR_UNSUPPORTED), (dict(x_dtype=2), drl.DR_ERR_UNSUPPORTED),
    (dict(res_dtype=-1), drl.DR_ERR_UNSUPPORTED), (dict(dy_dtype=7), drl.DR_ERR_UNSUPPORTED),
    (dict(eps=-1.0), drl.DR_ERR_UNSUPPORTED), (dict(eps=float("nan")), drl.DR_ERR_UNSUPPORTED),
    (dict(B=2 ** 20, H=2 ** 12), drl.DR_ERR_UNSUPPORTED), (dict(H=2 ** 20 + 1, L=1), drl.DR_ERR_UNSUPPORTED),
])
def test_norm_descriptors(kw, code):
    for f in (rf, re_, rb):
        assert f(rn(**kw)) == code and drl.dr_last_error()
    assert drl.dr_rmsnorm_bwd_workspace_bytes(rn(**kw)) == 0


def test_norm_arguments():
    for f in (rf, re_, rb):
        assert f(None) == drl.DR_ERR_NULL
    for n in ("x", "y"):
        assert rf(rn(), **{n: None}) == re_(rn(), **{n: None}) == drl.DR_ERR_NULL
    assert re_(rn(), scale=None) == drl.DR_ERR_NULL
    assert rf(rn(), residual=None) == rf(rn(), total=None) == drl.DR_ERR_NULL
    for n in ("x", "rstd", "dy", "dx"):
        assert rb(rn(), **{n: None}) == drl.DR_ERR_NULL
    assert rf(rn(x_dtype=drl.DR_F32, res_dtype=drl.DR_BF16)) == drl.DR_ERR_UNSUPPORTED
    assert re_(rn(block=64)) == drl.DR_ERR_UNSUPPORTED
    # alignment of one element
    for f, n, off in ((rf, "x", 1), (rf, "residual", 2), (rf, "total", 2), (rf, "weight", 2), (rf, "y", 1), (rf, "rstd", 2),
                      (re_, "scale", 2), (rb, "dy", 2), (rb, "ds", 1), (rb, "dx", 1), (rb, "dweight", 2), (rb, "ws", 8)):
        assert f(rn(), **{n: F(20) + off}) == drl.DR_ERR_ALIGN, (f, n)
    for n in ("x", "res", "y", "total"):
        d = rn()
        setattr(d, n, S(10, -5, 3))
        assert rf(d) == drl.DR_ERR_SHAPE
    for f, n in ((rf, "y"), (rf, "total"), (rb, "y")):
        d = rn()
        setattr(d, n, S(3 * 50 * 200, 50 * 200, 100))
        assert f(d) == drl.DR_ERR_UNSUPPORTED and "overlap" in drl.dr_last_error()


def test_norm_overlaps_and_workspace():
    for i, n in enumerate(RF[:3]):
        for o in ("y", "total", "rstd"):
            assert rf(rn(), **{o: F(i) + 256}) == drl.DR_ERR_UNSUPPORTED and "overlaps" in drl.dr_last_error()
    assert re_(rn(), scale=F(3) + 16) == drl.DR_ERR_UNSUPPORTED
    # the sum in the residual's place, but with other strides
    d = rn()
    d.total.b += 8
    assert rf(d, total=F(1)) == drl.DR_ERR_UNSUPPORTED and "overlaps" in drl.dr_last_error()
    assert rf(rn(), total=F(1) + 4) == drl.DR_ERR_UNSUPPORTED
    assert rf(rn(), total=F(1), rstd=F(0)) == drl.DR_ERR_UNSUPPORTED and "rstd" in drl.dr_last_error()   # goes on
    # the last byte of y, and the first one behind it
    size = 2 * 3 * 50 * 200
    assert re_(rn(), scale=F(3) + size - 4) == drl.DR_ERR_UNSUPPORTED
    need = drl.dr_rmsnorm_bwd_workspace_bytes(rn())
    assert need > 0
    for i, n in enumerate(RB[:7]):
        assert rb(rn(), wbytes=need - 1, ws=F(i) + 256) == drl.DR_ERR_UNSUPPORTED
        assert "workspace" in drl.dr_last_error()
    assert rb(rn(), wbytes=need - 1) == rb(rn(), ws=None) == drl.DR_ERR_WORKSPACE


# ---------------------------------------------------------------- convolution

def sc(**kw):
    base = dict(B=2, L=50, C=200, W=4, x_dtype=drl.DR_BF16, y_dtype=drl.DR_BF16, dy_dtype=drl.DR_F32, act=1)
    base.update(kw)
    L, C = base["L"], base["C"]
    return drl.ShortConvDesc(*base.values(), *(S(L * C, 0, C),) * 3)


CF = ("x", "weight", "bias", "state", "y", "state_out")
CB = ("x", "weight", "bias", "state", "dy", "dstate_out", "dx", "dweight", "dbias", "dstate", "ws")
CS = ("x", "weight", "bias", "state", "y")


def cf(d, **kw):
    return call("dr_short_conv_fwd", d, CF, kw)


def cb(d, wbytes=BIG, **kw):
    return call("dr_short_conv_bwd", d, CB, kw, wbytes)


def cs(d, **kw):
    return call("dr_short_conv_step", d, CS, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), drl.DR_ERR_SHAPE), (dict(L=-1), drl.DR_ERR_SHAPE), (dict(C=0), drl.DR_ERR_SHAPE),
    (dict(C=-3), drl.DR_ERR_SHAPE), (dict(W=1), drl.DR_ERR_UNSUPPORTED), (dict(W=9), drl.DR_ERR_UNSUPPORTED),
    (dict(act=2), drl.DR_ERR_UNSUPPORTED), (dict(x_dtype=3), drl.DR_ERR_UNSUPPORTED),
    (dict(y_dtype=-1), drl.DR_ERR_UNSUPPORTED), (dict(C=2 ** 24 + 1), drl.DR_ERR_UNSUPPORTED),
    (dict(L=2 ** 31 - 1), drl.DR_ERR_UNSUPPORTED), (dict(B=2 ** 31 - 1), drl.DR_ERR_UNSUPPORTED),
])
def test_conv_descriptors(kw, code):
    for f in (cf, cb, cs):
        assert f(sc(**kw)) == code and drl.dr_last_error()
    assert drl.dr_short_conv_bwd_workspace_bytes(sc(**kw)) == 0


def test_conv_arguments():
    for f in (cf, cb, cs):
        assert f(None) == drl.DR_ERR_NULL
    for f, names in ((cf, ("x", "weight", "y")), (cb, ("x", "weight", "dy", "dx")), (cs, ("x", "weight", "state", "y"))):
        for n in names:
            assert f(sc(), **{n: None}) == drl.DR_ERR_NULL
        for n in ("x", "state"):
            assert f(sc(), **{n: F(20) + 1}) == drl.DR_ERR_ALIGN
        for n in ("weight", "bias"):
            assert f(sc(), **{n: F(20) + 2}) == drl.DR_ERR_ALIGN
    for n in ("dy", "dstate_out", "dweight", "dbias", "dstate"):
        assert cb(sc(), **{n: F(20) + 2}) == drl.DR_ERR_ALIGN
    assert cb(sc(), ws=F(20) + 8) == drl.DR_ERR_ALIGN
    d = sc()
    d.x.t = -200
    assert cf(d) == cb(d) == drl.DR_ERR_SHAPE
    d = sc()
    d.y.t = 100
    assert cf(d) == cb(d) == drl.DR_ERR_UNSUPPORTED and "overlap" in drl.dr_last_error()
    # an enormous batch of long sequences
    assert cf(sc(B=2 ** 22, L=2 ** 30)) == drl.DR_ERR_UNSUPPORTED


def test_conv_overlaps_and_workspace():
    for i in range(4):
        assert cf(sc(), y=F(i) + 64) == drl.DR_ERR_UNSUPPORTED
    for i in range(3):
        assert cf(sc(), state_out=F(i) + 64) == drl.DR_ERR_UNSUPPORTED
    assert cf(sc(), state_out=F(3) + 2) == drl.DR_ERR_UNSUPPORTED      # inside the state, not the state itself
    assert cs(sc(), y=F(3) + 2) == drl.DR_ERR_UNSUPPORTED
    need = drl.dr_short_conv_bwd_workspace_bytes(sc())
    assert need > 0
    for i in range(10):
        assert cb(sc(), wbytes=need - 1, ws=F(i) + 256) == drl.DR_ERR_UNSUPPORTED
    assert cb(sc(), wbytes=need - 1) == cb(sc(), ws=None) == drl.DR_ERR_WORKSPACE


# ---------------------------------------------------------------- recurrence

def gs(**kw):
    base = dict(B=2, L=5000, C=200, x_dtype=drl.DR_BF16, gate_dtype=drl.DR_F32, h_dtype=drl.DR_F32, dh_dtype=drl.DR_BF16,
                grad_dtype=drl.DR_F32, decay=0, inputs=2)
    base.update(kw)
    L, C = base["L"], base["C"]
    return drl.GatedScanDesc(*base.values(), *(S(L * C, 0, C),) * 6)


GF = ("x", "gate", "h0", "h", "h_final", "ws")
GB = ("x", "gate", "h0", "h", "dh", "dh_final", "dx", "dgate", "dh0", "ws")
GS = ("x", "gate", "state", "h")


def gf(d, wbytes=BIG, **kw):
    return call("dr_gated_scan_fwd", d, GF, kw, wbytes)


def gb(d, wbytes=BIG, **kw):
    return call("dr_gated_scan_bwd", d, GB, kw, wbytes)


def gst(d, **kw):
    return call("dr_gated_scan_step", d, GS, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), drl.DR_ERR_SHAPE), (dict(L=-1), drl.DR_ERR_SHAPE), (dict(C=0), drl.DR_ERR_SHAPE),
    (dict(decay=2), drl.DR_ERR_UNSUPPORTED), (dict(inputs=3), drl.DR_ERR_UNSUPPORTED),
    (dict(inputs=-1), drl.DR_ERR_UNSUPPORTED), (dict(x_dtype=2), drl.DR_ERR_UNSUPPORTED),
    (dict(x_dtype=drl.DR_F32, gate_dtype=drl.DR_BF16), drl.DR_ERR_UNSUPPORTED),
    (dict(grad_dtype=5), drl.DR_ERR_UNSUPPORTED), (dict(dh_dtype=5), drl.DR_ERR_UNSUPPORTED),
    (dict(C=2 ** 24 + 1), drl.DR_ERR_UNSUPPORTED), (dict(L=2 ** 31 - 1), drl.DR_ERR_UNSUPPORTED),
    (dict(B=2 ** 31 - 1), drl.DR_ERR_UNSUPPORTED),
])
def test_scan_descriptors(kw, code):
    for f in (gf, gb, gst):
        assert f(gs(**kw)) == code and drl.dr_last_error()
    assert drl.dr_gated_scan_fwd_workspace_bytes(gs(**kw)) == drl.dr_gated_scan_bwd_workspace_bytes(gs(**kw)) == 0


def test_scan_arguments():
    for f in (gf, gb, gst):
        assert f(None) == drl.DR_ERR_NULL
    for f, names in ((gf, ("x", "gate", "h")), (gb, ("x", "gate", "h", "dh", "dx", "dgate")),
                     (gst, ("x", "gate", "state", "h"))):
        for n in names:
            assert f(gs(), **{n: None}) == drl.DR_ERR_NULL
    for f, n, off in ((gf, "x", 1), (gf, "gate", 2), (gf, "h0", 2), (gf, "h", 2), (gf, "h_final", 2), (gb, "dh", 1),
                      (gb, "dh_final", 2), (gb, "dx", 2), (gb, "dgate", 2), (gb, "dh0", 2), (gst, "state", 2)):
        assert f(gs(), **{n: F(20) + off}) == drl.DR_ERR_ALIGN, (f, n)
    for f, n in ((gf, "x"), (gf, "gate"), (gf, "h"), (gb, "dh"), (gb, "dx"), (gb, "dgate")):
        d = gs()
        setattr(d, n, S(-1, 0, 200))
        assert f(d) == drl.DR_ERR_SHAPE
    for f, n in ((gf, "h"), (gb, "dx"), (gb, "dgate")):
        d = gs()
        setattr(d, n, S(0, 0, 200))
        assert f(d) == drl.DR_ERR_UNSUPPORTED and "overlap" in drl.dr_last_error()


def test_scan_overlaps():
    for i in range(3):
        assert gf(gs(), h=F(i) + 64) == drl.DR_ERR_UNSUPPORTED
    assert gf(gs(), h_final=F(2) + 4) == drl.DR_ERR_UNSUPPORTED        # inside h0, not h0 itself
    assert gf(gs(), h_final=F(3) + 64) == drl.DR_ERR_UNSUPPORTED
    for i in range(6):
        for o in ("dx", "dgate", "dh0"):
            assert gb(gs(), **{o: F(i) + 64}) == drl.DR_ERR_UNSUPPORTED
    assert gb(gs(), dx=F(7) + 64) == drl.DR_ERR_UNSUPPORTED
    assert gst(gs(), h=F(2) + 4) == drl.DR_ERR_UNSUPPORTED
    for f, wsz, n in ((gf, drl.dr_gated_scan_fwd_workspace_bytes, 5), (gb, drl.dr_gated_scan_bwd_workspace_bytes, 9)):
        need = wsz(gs())
        if need:
            for i in range(n):
                assert f(gs(), wbytes=need - 1, ws=F(i) + 256) == drl.DR_ERR_UNSUPPORTED
            assert f(gs(), wbytes=need - 1) == f(gs(), ws=None) == drl.DR_ERR_WORKSPACE
            assert f(gs(), ws=F(20) + 8) == drl.DR_ERR_ALIGN


def test_nothing_to_do():
    assert rf(rn(B=0)) == rb(rn(L=0), dweight=None, ws=None) == drl.DR_OK
    assert cf(sc(B=0)) == cs(sc(B=0)) == gf(gs(B=0)) == gst(gs(B=0)) == drl.DR_OK
    assert cf(sc(L=0), state_out=None) == gf(gs(L=0), h_final=None) == gb(gs(L=0), dh0=None) == drl.DR_OK
    assert cf(sc(L=0), state_out=F(3)) == gf(gs(L=0), h_final=F(2)) == drl.DR_OK     # in place: nothing moves
    assert drl.dr_rmsnorm_bwd_workspace_bytes(rn(L=0)) == drl.dr_short_conv_bwd_workspace_bytes(sc(L=0)) == 0


def test_sizes_past_31_bits_are_refused_by_the_binding():
    for plan, sizes in ((drl._short_conv_plan, (2 ** 31, 1, 8, 4, 0, 0, 0, 0)),
                        (drl._gated_scan_plan, (False, (1, 2 ** 32 + 4, 8, 0, 0, 0, 0, 0, 0, 0))),
                        (drl._rmsnorm_plan, (1, 1, 2 ** 31, 8, 0, 0, 0, 0, 0, 1e-5, 0))):
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            plan(*sizes) if isinstance(sizes[0], bool) else plan(sizes)


# ---------------------------------------------------------------- the oracle

def grads(f, inputs, cotangents):
    leaves = [t.clone().requires_grad_() for t in inputs]
    out = f(*leaves)
    return torch.autograd.grad(sum((o * c).sum() for o, c in zip(out, cotangents)), leaves)


def test_oracle_gradients():
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, res, w, dy, ds = r(6, 9), r(6, 9), r(9), r(6, 9), r(6, 9)
    want = grads(lambda x, res, w: ref.rms_forward(x, res, w, 1e-3)[:2], (x, res, w), (ds, dy))
    s, _, rstd = ref.rms_forward(x, res, w, 1e-3)
    dx, terms = ref.rms_backward(s, w, rstd, dy, ds)
    for got, v in zip((dx, dx, terms.sum(0)), want):
        assert torch.allclose(got, v, rtol=1e-12, atol=1e-12)
    x, w, b, st, dy, dl = r(2, 7, 3), r(3, 4), r(3), r(2, 3, 3), r(2, 7, 3), r(2, 3, 3)
    for silu in (False, True):
        for L in (1, 2, 7):
            want = grads(lambda x, w, b, st: ref.conv_forward(x, w, b, st, silu)[:2], (x[:, :L], w, b, st), (dy[:, :L], dl))
            got = ref.conv_backward(x[:, :L], w, b, st, dy[:, :L], dl, silu)
            for n, v in zip(("dx", "dweight", "dbias", "dstate"), want):
                assert torch.allclose(got[n], v, rtol=1e-11, atol=1e-11), (n, silu, L)
    x, g, h0, dh, dl = r(2, 9, 3), -r(2, 9, 3).abs() - 0.01, r(2, 3), r(2, 9, 3), r(2, 3)
    for decay in ("log", "logit"):
        for inputs in ("plain", "blend", "unit"):
            want = grads(lambda x, g, h0: ref.scan_forward(x, g, h0, decay, inputs), (x, g, h0), (dh, dl))
            h, _ = ref.scan_forward(x, g, h0, decay, inputs)
            got = ref.scan_backward(x, g, h0, h, dh, dl, decay, inputs)
            for n, v in zip(("dx", "dgate", "dh0"), want):
                assert torch.allclose(got[n], v, rtol=1e-10, atol=1e-10), (n, decay, inputs)


def test_wrong_results_do_not_pass():
    """The bounds see a lost carry, a shifted tap, a missing factor and a scale that is
    one power of two off."""
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, g, h0 = r(1, 40, 4), -r(1, 40, 4).abs(), r(1, 4)
    h, _ = ref.scan_forward(x, g, h0, "log", "unit")
    e, _ = ref.scan_errors(x, g, h0, "log", "unit")
    for wrong in (ref.scan_forward(x, g, None, "log", "unit")[0], ref.scan_forward(x, g, h0, "log", "blend")[0],
                  ref.scan_forward(x, g.roll(1, 1), h0, "log", "unit")[0]):
        with pytest.raises(AssertionError):
            ref.near(wrong.float(), h, e, "h")
    ref.near(h.float(), h, e, "h")
    w = r(4, 4)
    y = ref.conv_forward(x, w, None, None, True)
    _, b = ref.conv_bounds(x, w, None, None, True, y)
    with pytest.raises(AssertionError):
        ref.near(ref.conv_forward(x, w.roll(1, 1), None, None, True)[0].bfloat16(), y[0], b, "y")
    ref.near(y[0].bfloat16(), y[0], b, "y")
    v = torch.tensor([1.0, 3.1, 447.0, 2.0 ** -9, 2.0 ** -6, 17.0], dtype=torch.float64)
    assert ref.e4m3_step(v).tolist() == [0.125, 0.25, 32.0, 2.0 ** -9, 2.0 ** -9, 2.0]
