"""How exact the gated linear recurrence is on the GPU where single roundings would be
multiplied: strong decays, and memories of very many tokens (u = 2^-24)."""
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


def one_token(gate, h0, x, **m):
    """h of one token from the forward, from the step, and from the gradient of h0 or x."""
    import delta_rule_linear_amd as drl
    g, s = gate[None], torch.full((1, gate.numel()), h0, device="cuda")
    x = torch.full_like(g, x)
    h = drl.dr_gated_scan_fwd(x[None], g[None], s, **m)[0]
    back = drl.dr_gated_scan_bwd(x[None], g[None], s, h, torch.ones_like(h), **m)
    step = drl.dr_gated_scan_step(s.clone(), x, g, **m)
    return h[0, 0], step[0], back["dh0"][0] if h0 else back["dx"][0, 0]


def units(got, want):
    return ((d(got) - want).abs() / want) / U


STRONG = -torch.cat([torch.linspace(0.41, 87.0, 20011), torch.tensor([5.0, 20.0, 60.0, 87.0])])


def test_strong_decays_relative_to_themselves():
    """e^g: the exponential itself is off by a unit in the last place (2 u), the correction of
    its argument is rounded once (u) and takes ln 2 in 24 bits (off by 1.91e-9, times |g| log2 e: 0.047 |g|
    u).  The sigmoid besides: 1 + e^g (the same, half of it at most, and u), its reciprocal (2 u), the
    product (u)."""
    announce("strong decays")
    g = STRONG.cuda()
    e = 3.1 + 0.047 * d(g).abs()
    for h in one_token(g, 1.0, 0.0, decay="log"):
        assert (units(h, d(g).exp()) <= e).all()
    for h in one_token(g, 1.0, 0.0, decay="logit"):
        assert (units(h, torch.sigmoid(d(g))) <= 1.5 * e + 4.1).all()


def test_inputs_of_long_memories():
    """1 - a, of logits whose a is near one, as exact as the sigmoid; of strong decays 1 - e^g,
    with e^g / (1 - e^g) below 2.1 of e^g's error, and u."""
    announce("inputs of long memories")
    g = -STRONG.cuda()
    e = 3.1 + 0.047 * d(g).abs()
    for h in one_token(g, 0.0, 1.0, decay="logit", inputs="blend"):
        assert (units(h, torch.sigmoid(-d(g))) <= 1.5 * e + 4.1).all()
    for h in one_token(-g, 0.0, 1.0, decay="log", inputs="blend"):
        assert (units(h, -torch.expm1(-d(g))) <= 2.1 * e + 1.1).all()


def test_strong_decays_over_tokens():
    """Four tokens of about e^-20: each as above (4.1 u), and a rounding of the state each."""
    import delta_rule_linear_amd as drl
    announce("strong decays over tokens")
    g = torch.linspace(-21.8, -19.0, 1024, device="cuda").expand(1, 4, 1024).contiguous()
    x, one = torch.zeros_like(g), torch.ones((1, 1024), device="cuda")
    h, last = drl.dr_gated_scan_fwd(x, g, one, decay="log")
    for t in range(4):
        assert (units(h[0, t], d(g)[0, :t + 1].sum(0).exp()) <= 5.2 * (t + 1)).all()
    assert torch.equal(last[0], h[0, 3])
    back = drl.dr_gated_scan_bwd(x, g, one, h, x, one, decay="log")
    assert (units(back["dh0"][0], d(g)[0].sum(0).exp()) <= 5.2 * 4).all()


@pytest.mark.parametrize("gate,B,L,C", [(-1e-6, 1, 2 ** 20, 8), (-1.3e-7, 1, 2 ** 20, 72), (-1e-6, 3, 2 ** 20 - 77, 5),
                                        (-2.0 ** -14, 1, 200000, 8)])
@pytest.mark.parametrize("inputs", ["plain", "blend"])
def test_memories_of_very_many_tokens(gate, B, L, C, inputs):
    """The same decay and input for 2^20 tokens, 8192 tiles: a decay rounded to 24 bits anywhere on
    the way would be the same error in every tile, a part in 14000 of the state at -1e-6.  The state itself is
    rounded a few times in each tile, at random, and forgets 8192 tiles over 1e6 tokens: about the root of 3 x 8192 of
    2^-24, below 1e-5."""
    import delta_rule_linear_amd as drl
    announce("memories of very many tokens", gate, B, L, C, inputs)
    g, x = torch.full((B, L, C), gate, device="cuda"), torch.ones((B, L, C), device="cuda")
    m = dict(decay="log", inputs=inputs)
    h, last = drl.dr_gated_scan_fwd(x, g, None, **m)
    rest = -torch.expm1(g[0, 0, 0].double().cpu())
    t = torch.tensor([L, L // 2, L // 3, 4097, 128, 1], dtype=torch.float64)
    geometric = -torch.expm1(t * g[0, 0, 0].double().cpu()) / rest    # the sum of a^k over t tokens
    want = geometric * (1 if inputs == "plain" else rest)
    for k, w in zip(t.long().tolist(), want):
        assert float((d(h[:, k - 1]) / w - 1).abs().max()) <= 1e-5, k
    assert torch.equal(last, h[:, -1])
    # the gradient runs through the same maps, backwards
    one = torch.ones_like(h)
    back = drl.dr_gated_scan_bwd(x, g, None, h, one, decay="log")
    for k, w in zip(t.long().tolist(), geometric):
        assert float((d(back["dx"][:, L - k]) / w - 1).abs().max()) <= 1e-5, k
