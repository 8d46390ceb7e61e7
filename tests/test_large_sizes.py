"""Sizes past 31 bits are refused by the binding: a C int would keep their low
bits, and the call would take the first few rows for all of them."""
import pytest

import delta_rule_linear_amd as drl

torch = pytest.importorskip("torch")

BIG = 2 ** 32 + 3
S0 = (0, 0, 0)


@pytest.mark.parametrize("at", range(6))
def test_sizes_of_attention_descriptors(at):
    sizes = [1, 2, 2, 5, 8, 8]
    sizes[at] = BIG
    with pytest.raises(ValueError, match="2\\^31"):
        drl.linattn_desc(*sizes, drl.DR_BF16, drl.DR_F32, "none")
    for bwd, n in ((False, 4), (True, 7)):
        with pytest.raises(ValueError, match="2\\^31"):
            drl._linattn_plan(bwd, (*sizes, drl.DR_BF16, drl.DR_F32, 0), *[S0] * n)


def test_sizes_of_steps_and_norms():
    with pytest.raises(ValueError, match="2\\^31"):
        drl._linattn_step_plan(BIG, 1, 1, 8, 8, drl.DR_BF16, drl.DR_F32, 0)
    for at in range(4):
        sizes = [1, 1, 5, 8]
        sizes[at] = BIG
        with pytest.raises(ValueError, match="2\\^31"):
            drl._layernorm_plan((*sizes, 0, 1, 1, 1, 1e-5), S0, S0)


@pytest.mark.gpu
def test_a_call_of_more_tokens():
    """Broadcast rows (stride 0) reach such lengths in any memory."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.ones((1, 1, 1, 8), dtype=torch.bfloat16, device="cuda").expand(1, 1, BIG, 8)
    o = torch.zeros((1, 1, 1, 8), device="cuda").expand(1, 1, BIG, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        drl.dr_linear_attn_fwd(x, x, x, decay="none", o=o)
    assert not o[0, 0, 0].any()


def test_other_numbers_are_not_sizes():
    """eps is checked by the library, which refuses an infinite one."""
    import ctypes
    desc, _, _ = drl._layernorm_plan((1, 1, 5, 8, 0, 1, 1, 1, float("inf")), S0, S0)
    p = [0x7f0000000000 + (i << 36) for i in range(6)]
    assert drl.lib().dr_layernorm_fwd(ctypes.byref(desc), *p, None) == drl.DR_ERR_UNSUPPORTED
    assert "eps" in drl.dr_last_error()
