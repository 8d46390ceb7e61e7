"""The RMS norm, the short convolution and the gated recurrence at the limits of their
sizes, without a GPU: what is too large is refused before any device work."""
import pytest

import delta_rule_linear_amd as drl

pytest.importorskip("torch")
from test_seqops_cpu import cb, cf, cs, gb, gf, gs, gst, sc  # noqa: E402


@pytest.mark.parametrize("B,C", [(2 ** 30, 8), (2 ** 30 + 1, 8), (2 ** 31 - 1, 8), (2 ** 30, 2 ** 23), (2 ** 29, 129),
                                 (2 ** 14, 2 ** 23)])
def test_batches_past_31_bits_are_refused(B, C):
    """B ceil(C / 128) reaches 2^30; twice B alone is no 32-bit number from 2^30 on."""
    for f, desc in ((cf, sc), (cb, sc), (cs, sc), (gf, gs), (gb, gs), (gst, gs)):
        assert f(desc(B=B, C=C, L=1)) == drl.DR_ERR_UNSUPPORTED and "too large" in drl.dr_last_error()
    for f, desc in ((drl.dr_short_conv_bwd_workspace_bytes, sc), (drl.dr_gated_scan_fwd_workspace_bytes, gs),
                    (drl.dr_gated_scan_bwd_workspace_bytes, gs)):
        assert f(desc(B=B, C=C, L=1)) == 0


def test_the_largest_batch_is_taken():
    assert drl.dr_short_conv_bwd_workspace_bytes(sc(B=2 ** 30 - 1, C=8, L=1)) > 0
    assert drl.dr_short_conv_bwd_workspace_bytes(sc(B=2 ** 29 - 1, C=129, L=1)) > 0
    # with many columns a workgroup walks whole sequences: no workspace, and no complaint
    assert drl.dr_gated_scan_fwd_workspace_bytes(gs(B=2 ** 30 - 1, C=8, L=1)) == 0
    assert gf(gs(B=2 ** 30 - 1, C=8, L=1), x=None) == drl.DR_ERR_NULL


def test_scan_workspaces_are_needed_and_checked():
    """Long sequences of few columns need one, forward and backward alike (both cut them into
    the same tiles)."""
    need = drl.dr_gated_scan_fwd_workspace_bytes(gs())
    assert need > 0 and need == drl.dr_gated_scan_bwd_workspace_bytes(gs())
    for f in (gf, gb):
        assert f(gs(), wbytes=need - 1) == f(gs(), ws=None) == drl.DR_ERR_WORKSPACE
    # one tile, or columns enough
    for kw in (dict(L=128), dict(B=1024, L=129, C=8)):
        assert drl.dr_gated_scan_fwd_workspace_bytes(gs(**kw)) == drl.dr_gated_scan_bwd_workspace_bytes(gs(**kw)) == 0
    assert drl.dr_gated_scan_fwd_workspace_bytes(gs(L=129)) > 0
