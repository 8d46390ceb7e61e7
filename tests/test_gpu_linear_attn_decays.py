"""How exact the decays themselves are, on the GPU: inputs that leave nothing else
in the outputs.  u = 2^-24."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def decays(decay, H, L, x, seed):
    """log alpha whose sum over the tokens is about x."""
    gen = torch.Generator().manual_seed(seed)
    shape = (H,) if decay == "head" else (1, H, L)
    return x / L * (0.5 + torch.rand(shape, generator=gen))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("L,x", [(64, -75.0), (64, -1.0), (130, -70.0), (500, -75.0), (2000, -60.0)])
def test_decays_of_states(L, x, decay, dtype):
    """k = 0, S0 = 1 and one-hot q: o_t = e^{u_t} and S_L = e^{u_L}, whatever the size
    of u.  An exponential is off by 4 u (two of the hardware's, one of the factor for
    the exponent's low part, one of their product) and its use by one more, in
    every chunk (or segment) before; bf16 adds up three terms of the state, 2 u."""
    import delta_rule_linear_amd as drl
    announce("decays of states", L, x, decay, dtype)
    H, D = 3, 64
    la = decays(decay, H, L, x, L)
    q = torch.zeros(1, H, L, D)
    q[..., 5] = 1
    v = torch.randn((1, H, L, D), generator=torch.Generator().manual_seed(1))
    t = lambda a: a.to(DT[dtype]).cuda()  # noqa: E731
    S0 = torch.ones(1, H, D, D).cuda()
    o, S = drl.dr_linear_attn_fwd(t(q), t(0 * q), t(v), la.cuda(), S0, decay=decay)
    a = la.double() if decay == "token" else la.double()[None, :, None].expand(1, H, L)
    want = a.cumsum(-1).exp()[..., None]
    chunk = (torch.arange(L) // 64).double()[:, None]
    # below 2^-126 fp32 has no normal values: a result there may be zero
    for got, exact, c, what in ((o, want, chunk, "o"), (S, want[:, :, -1:], chunk[-1], "S")):
        err = ((got.double().cpu() - exact).abs() - 2.0 ** -126).clamp(min=0) / exact
        assert bool((err <= (5 * c + 8) * U).all()), f"{what}: {float((err / U).max()):.3g} u"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("x", [-1.0, -20.0, -75.0])
def test_decays_between_tokens(x, dtype):
    """One k of a chunk is not zero: o_i = e^{x} with x the log alphas behind it.
    The difference of two fp32 exponents is rounded twice, 2 |x| u, the exponential
    off by 2 u, and three products and sums by one each (bf16: two terms more)."""
    import delta_rule_linear_amd as drl
    announce("decays between tokens", x, dtype)
    H, L, D, j = 2, 64, 64, 3
    la = decays("token", H, L, x, 7)
    q = torch.zeros(1, H, L, D)
    q[..., 5] = 1
    k = torch.zeros(1, H, L, D)
    k[:, :, j, 5] = 1
    t = lambda a: a.to(DT[dtype]).cuda()  # noqa: E731
    o, S = drl.dr_linear_attn_fwd(t(q), t(k), t(torch.ones(1, H, L, D)), la.cuda(), decay="token")
    a = la.double().cumsum(-1)
    e = (a - a[:, :, j:j + 1])[:, :, j:]
    err = (o.double().cpu()[:, :, j:] - e.exp()[..., None]).abs() / e.exp()[..., None]
    assert bool((err <= (2 * e.abs() + 8)[..., None] * U).all()), f"{float((err / U).max()):.3g} u"
    assert not o[:, :, :j].any()
    # the state's: 4 u and its use
    err = (S[:, :, 5].double().cpu() - e[:, :, -1:].exp()).abs() / e[:, :, -1:].exp()
    assert bool((err <= 8 * U).all()), f"S: {float((err / U).max()):.3g} u"


@pytest.mark.parametrize("dtype,e", [("bf16", 120), ("bf16", -100), ("f32", 120), ("f32", -116)])
def test_magnitudes(dtype, e):
    """v and S0 scaled by 2^e (to 2^126 in the state): every 2-norm within the
    expected size, 8 standard deviations of n roundings, as in linattn_ref.check."""
    import delta_rule_linear_amd as drl
    import linattn_ref as ref
    announce("magnitudes", dtype, e)
    gen = torch.Generator().manual_seed(3)
    L, D = 100, 64
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k = (r(1, 1, L, D).to(DT[dtype]) for _ in range(2))
    q = q * 2.0 ** -8
    v, S0 = (r(1, 1, L, D) * 2.0 ** (e - 4)).to(DT[dtype]), r(1, 1, D, D) * 2.0 ** (e - 2)
    la = -0.1 * torch.rand((1, 1, L), generator=gen)
    o, S = drl.dr_linear_attn_fwd(q.cuda(), k.cuda(), v.cuda(), la.cuda(), S0.cuda(), decay="token")
    wo, wS = ref.forward(q.double(), k.double(), v.double(), la.double().exp(), S0.double())
    n = L + 2 * D + 256
    for got, want in ((o, wo), (S, wS)):
        assert bool(torch.isfinite(got).all())
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= 8 * n ** 0.5 * U, err


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_roundings_of_a_long_state(dtype):
    """S_L = sum of k v^T over 64 chunks without a decay, in one segment.  A rounding
    to nearest is off by 0.425 u of the value, root mean square over mantissas; S
    grows like the square root of the tokens, so r of them in each of N chunks make
    0.425 u sqrt(r N / 2) of S_L.  fp32: 32 tokens are summed at a time, r = 2 and
    3.4 u, which those sums, small against S_L, bring to 3.8 u at most.  bf16: each
    instruction takes 32 tokens and one of z's three terms, r = 6 and 5.9 u.  Half
    as much again is allowed."""
    import delta_rule_linear_amd as drl
    announce("roundings of a long state", dtype)
    B, H, L, D = 8, 64, 4096, 8
    d = drl.linattn_desc(B, H, H, L, D, D, drl.DR_F32, drl.DR_F32, "none")
    assert drl.dr_linear_attn_fwd_workspace_bytes(d) == 0   # one segment
    gen = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn((B, H, L, D), generator=gen).to(DT[dtype]) for _ in range(3))
    _, S = drl.dr_linear_attn_fwd(q.cuda(), k.cuda(), v.cuda(), decay="none")
    want = k.double().transpose(2, 3).contiguous() @ v.double()
    err = float((S.double().cpu() - want).norm() / want.norm())
    assert err <= 1.5 * (3.8 if dtype == "f32" else 5.9) * U, f"{err / U:.3g} u"
