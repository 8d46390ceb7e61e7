"""A workspace that shares memory with an input is refused (it is written while
the input is read), without a GPU.  With a size that is too small by one the calls
below would stop at the next check."""
import pytest

import delta_rule_linear_amd as drl
from test_linear_attn_cpu import BNAMES, F, NAMES, bwd, desc, fwd, ln, lnb

pytest.importorskip("torch")


@pytest.mark.parametrize("name", [n for n in NAMES if n != "ws"])
def test_forward(name):
    need = drl.dr_linear_attn_fwd_workspace_bytes(desc())
    assert fwd(desc(), wbytes=need - 1, ws=F(NAMES.index(name)) + 256) == drl.DR_ERR_UNSUPPORTED
    assert "workspace" in drl.dr_last_error() and "overlaps" in drl.dr_last_error()
    assert fwd(desc(), wbytes=need - 1) == drl.DR_ERR_WORKSPACE


@pytest.mark.parametrize("name", [n for n in BNAMES if n != "ws"])
def test_backward(name):
    need = drl.dr_linear_attn_bwd_workspace_bytes(desc())
    assert bwd(desc(), wbytes=need - 1, ws=F(BNAMES.index(name)) + 256) == drl.DR_ERR_UNSUPPORTED
    assert "workspace" in drl.dr_last_error() and "overlaps" in drl.dr_last_error()
    assert bwd(desc(), wbytes=need - 1) == drl.DR_ERR_WORKSPACE


@pytest.mark.parametrize("i,name", enumerate(("x", "w", "mean", "rstd", "dy", "dx", "dw", "db")))
def test_norm_backward(i, name):
    need = drl.dr_layernorm_bwd_workspace_bytes(ln())
    assert lnb(ln(), wbytes=need - 1, ws=F(i) + 256) == drl.DR_ERR_UNSUPPORTED
    assert "workspace" in drl.dr_last_error() and "overlaps" in drl.dr_last_error()
    assert lnb(ln(), wbytes=need - 1) == drl.DR_ERR_WORKSPACE


def test_a_workspace_that_is_not_needed():
    """No sums wanted, no segments: nothing is written there."""
    one = desc(B=128)
    assert drl.dr_linear_attn_fwd_workspace_bytes(one) == 0
    assert fwd(one, ws=F(0), o=F(6) + 256) == drl.DR_ERR_UNSUPPORTED   # o and S_final: the workspace itself passes
    assert "workspace" not in drl.dr_last_error()
