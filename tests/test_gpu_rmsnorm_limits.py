"""The RMS norm on either side of the largest rows that it takes: squares that sum to 2^128."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from seqops_ref import U, d  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


@pytest.mark.parametrize("D", [3, 64, 100, 1024, 2048, 2056, 8192, 16384])
@pytest.mark.parametrize("rows", [2, 3000])
def test_rows_of_large_values(D, rows):
    """Rows of one value all over and of a single large one, below and above the limit.  Below
    it rstd is off by the D roundings of the sum (half of each in the root) and a few more, y by one more."""
    import delta_rule_linear_amd as drl
    announce("large rows", D, rows)
    even = (2.0 ** 128 / D) ** 0.5          # D squares of this sum to 2^128
    x = torch.zeros((rows, D))
    x[0] = 0.99 * even
    x[1] = 1.01 * even
    if rows > 2:
        x[2, 0], x[3, D - 1] = 0.99 * 2.0 ** 64, 1.01 * 2.0 ** 64
        x[4, D // 2] = 1.2 * 2.0 ** 63
    x = x.cuda()
    y, rstd, _ = drl.dr_rmsnorm_fwd(x)
    y8, scale, rstd8, _ = drl.dr_rmsnorm_fwd_e4m3(x)
    assert torch.equal(rstd, rstd8)
    for r, over in ((0, False), (1, True), (2, False), (3, True), (4, False))[:5 if rows > 2 else 2]:
        if over:
            assert rstd[r] == 0 and not y[r].any() and not y8[r].float().any()
            assert not drl.dr_rmsnorm_bwd(x[r:r + 1], None, rstd[r:r + 1], torch.ones_like(x[r:r + 1]))["dx"].any()
        else:
            want = (d(x[r]).square().mean() + 1e-5).rsqrt()
            bound = (0.5 * D + 6) * U
            assert abs(float(d(rstd[r]) / want) - 1) <= bound
            assert ((d(y[r]) - d(x[r]) * want).abs() <= (bound + 2 * U) * (d(x[r]) * want).abs()).all()


def test_a_residual_counts_with_the_sum():
    import delta_rule_linear_amd as drl
    x = torch.full((2, 512), 2.0 ** 59, device="cuda")      # 512 squares of 2^59 are 2^127, of twice that 2^129
    y, rstd, total = drl.dr_rmsnorm_fwd(x, None, torch.stack([torch.zeros_like(x[0]), x[0]]))
    assert abs(float(rstd[0]) * 2.0 ** 59 - 1) <= 8 * U and (y[0] - 1).abs().max() <= 8 * U
    assert rstd[1] == 0 and not y[1].any() and torch.equal(total[1], 2 * x[0])
