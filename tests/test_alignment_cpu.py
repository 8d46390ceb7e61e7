"""Which addresses the layer norm and the linear attention take, without a GPU:
a call with accepted addresses goes on to the next check (an overlap or a missing
workspace), and the fake pointers are never touched."""
import pytest

import delta_rule_linear_amd as drl
from test_linear_attn_cpu import F, bwd, desc, fwd, ln, lnb, lnf

pytest.importorskip("torch")

FWD = ("x", "w", "b", "y", "mean", "rstd")
BWD = ("x", "w", "mean", "rstd", "dy", "dx", "dw", "db")
SIZE = {"x": 2, "dy": 2}   # ln()'s types: bf16 x and dy, fp32 y and dx


def at(name, off):
    """An address of the range that `name` usually has, `off` bytes on."""
    return {name: F(40) + off}


def f_next(d, **kw):
    """The forward's status behind the alignment check: y overlaps the bias."""
    p = {"b": F(50), "y": F(50), **kw}
    if "b" in kw:
        p["y"] = kw["b"] + (-kw["b"]) % 16
    if "y" in kw:
        p["b"] = kw["y"] - kw["y"] % 16
    return lnf(d, **p)


def test_norm_rows_of_any_width_start_anywhere():
    odd, even = ln(D=1001), ln(D=100)
    pad = ln(D=128)
    for f in ("x", "y", "dy"):   # 128 values of rows 131 apart
        setattr(pad, f, drl.Strides(4 * 100 * 131, 100 * 131, 131))
    for d in (odd, even, pad):
        for n in FWD:
            e = SIZE.get(n, 4)
            assert f_next(d, **at(n, e)) == drl.DR_ERR_UNSUPPORTED, n
            assert f_next(d, **at(n, 3 * e)) == drl.DR_ERR_UNSUPPORTED, n
            for off in {1, e - 1, e + e // 2}:
                assert f_next(d, **at(n, off)) == drl.DR_ERR_ALIGN, (n, off)
        for n in BWD:
            e = SIZE.get(n, 4)
            assert lnb(d, ws=None, **at(n, e)) == drl.DR_ERR_WORKSPACE, n
            for off in {1, e - 1, e + e // 2}:
                assert lnb(d, ws=None, **at(n, off)) == drl.DR_ERR_ALIGN, (n, off)
        assert lnb(d, ws=F(41) + 8) == drl.DR_ERR_ALIGN


def test_norm_statistics_of_a_slice():
    """Rows that are whole 16-byte pieces keep the general rule, but for what the
    backward reads one value per row of."""
    d = ln()
    for n in ("mean", "rstd"):
        assert lnb(d, ws=None, **at(n, 4)) == drl.DR_ERR_WORKSPACE
        assert lnb(d, ws=None, **at(n, 2)) == drl.DR_ERR_ALIGN
    for n in ("x", "w", "dy", "dx", "dw", "db"):
        assert lnb(d, ws=None, **at(n, 8)) == drl.DR_ERR_ALIGN
    for n in FWD:
        assert f_next(d, **at(n, 8)) == drl.DR_ERR_ALIGN


@pytest.mark.parametrize("kw,ok", [(dict(decay="head"), True), (dict(decay="token", L=4999), True),
                                   (dict(decay="token", L=5000), False)])
def test_decays(kw, ok):
    """A layer's row of a table [layers][heads], a sequence of a batch of any length."""
    d = desc(**kw)
    after = drl.DR_ERR_WORKSPACE if ok else drl.DR_ERR_ALIGN
    assert fwd(d, ws=None, la=F(40) + 4) == bwd(d, ws=None, la=F(40) + 4) == after
    assert bwd(d, ws=None, dla=F(40) + 12) == after
    for off in (1, 2, 6):
        assert fwd(d, ws=None, la=F(40) + off) == bwd(d, ws=None, dla=F(40) + off) == drl.DR_ERR_ALIGN


def test_step_decay():
    import ctypes
    S = drl.LinAttnStepDesc(N=4, H=6, Hk=3, Dk=64, Dv=128, in_dtype=1, out_dtype=0, decay=1)
    call = lambda la: drl.lib().dr_linear_attn_step(ctypes.byref(S), F(0), F(1), F(2), la, F(4), F(4), None)  # noqa: E731
    assert call(F(3) + 4) == drl.DR_ERR_UNSUPPORTED   # o overlaps S: the next check
    assert call(F(3) + 2) == drl.DR_ERR_ALIGN
