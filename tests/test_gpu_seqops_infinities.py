"""Infinities and NaN in the short convolution's backward on the GPU: they reach the
gradients that they are a part of, and no others."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seqops_ref as ref  # noqa: E402
from seqops_ref import DT, U, d, near  # noqa: E402

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def agree(got, want, bound, what):
    """The same infinities and NaN in the same places, and the others within the bound."""
    g = d(got)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what + ": NaN"
    ends = torch.isinf(want)
    assert torch.equal(torch.isinf(g), ends) and torch.equal(g[ends], want[ends]), what + ": infinities"
    ok = torch.isfinite(want)
    near(got.cpu()[ok], want[ok], bound.expand(want.shape)[ok], what)


# lengths that end on a step of the kernel's (a multiple of W, of four for two taps) and between two
@pytest.mark.parametrize("W,L", [(4, 8), (4, 9), (4, 64), (4, 259), (2, 8), (2, 7), (3, 12), (3, 13), (5, 51), (8, 16), (8, 85)])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("dtype,C", [("f32", 13), ("bf16", 16), ("bf16", 5)])
def test_convolution_backward(W, L, act, dtype, C):
    """One value that is infinite, or NaN, in the last tokens of a channel.  Tokens behind
    the last have no gradient, whatever the taps make of the rows before them."""
    import delta_rule_linear_amd as drl
    announce("convolution backward, infinities", W, L, act, dtype, C)
    gen = torch.Generator().manual_seed(W * 1000 + L)
    x = torch.randn((2, L, C), generator=gen).to(DT[dtype])
    dy = torch.randn((2, L, C), generator=gen).to(DT[dtype])
    w = torch.randn((C, W), generator=gen).abs() + 0.25
    w[:, 1::2] *= -1                                         # neighbouring taps of opposite signs
    b = torch.randn(C, generator=gen)
    clean = x.clone()
    for c, (back, v) in enumerate([(1, INF), (1, -INF), (1, NAN), (min(2, L), INF), (min(W, L), -INF)][:C]):
        x[0, L - back, c], clean[0, L - back, c] = v, 0.0
    g = drl.dr_short_conv_bwd(x.cuda(), w.cuda(), b.cuda(), None, dy.cuda(), activation=act, grad_dtype=torch.float32)
    x, clean, dy, w, b = (d(t) for t in (x, clean, dy, w, b))
    past = torch.cat([x.new_zeros(2, W - 1, C), x], 1)
    _, _, z = ref.conv_forward(x, w, b, None, False)
    # the slope of SiLU is 1 and 0 at the infinities
    zb = z.clamp(-1e4, 1e4)
    s = torch.sigmoid(zb)
    dz = dy * s * (1 + zb * (1 - s)) if act == "silu" else dy
    dz_err = torch.zeros_like(dz)
    if act == "silu":
        ez, _ = ref.conv_bounds(clean, w, b, None, True, ref.conv_forward(clean, w, b, None, True))
        dz_err = dy.abs() * (0.5 * ez + (12 + 4 * zb.abs()) * U * s * (1 + zb.abs() * (1 - s)))
        dz_err = torch.where(torch.isfinite(z), dz_err, 0 * dy)
    dx, mag, dw, bw = torch.zeros_like(past), torch.zeros_like(past), torch.zeros_like(w), torch.zeros_like(w)
    n = 2 * L + 8
    for j in range(W):
        dx[:, j:j + L] += w[:, j] * dz
        mag[:, j:j + L] += w[:, j].abs() * (dz_err + (W + 3) * U * dz.abs())
        dw[:, j] = (dz * past[:, j:j + L]).sum((0, 1))
        bw[:, j] = ((dz_err + n * U * dz.abs()) * past[:, j:j + L].abs()).sum((0, 1))
    agree(g["dx"], dx[:, W - 1:], mag[:, W - 1:], "dx")
    agree(g["dstate"], dx[:, :W - 1], mag[:, :W - 1], "dstate")
    agree(g["dweight"], dw, bw, "dweight")
    agree(g["dbias"], dz.sum((0, 1)), (dz_err + n * U * dz.abs()).sum((0, 1)), "dbias")
