"""Calls whose work would pass 2^32 threads in one launch dimension (a launch
holds fewer): many heads in the layer norm's weight sums, many small states in
the one-token step.  The results are compared on the GPU, in float64 where they
are rounded."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


@pytest.mark.parametrize("H,D", [(65536, 1024), (4096, 16384)])
def test_norm_weight_sums_of_many_heads(H, D):
    """H ceil(2 D / 32) tiles of 1024 threads: 2^32 threads.  One row per head, so
    that dbias is dy itself, and dweight dy (x - mean) rstd (three roundings)."""
    import delta_rule_linear_amd as drl
    announce("layer norm backward", H, D)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn((1, H, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.ones((H, D), device="cuda")
    _, mean, rstd = drl.dr_layernorm_fwd(x, w)
    g = drl.dr_layernorm_bwd(x, w, mean, rstd, dy)
    assert torch.equal(g["dbias"], dy[0].float())
    want = dy[0].double() * ((x[0].double() - mean[0].double()[:, None]) * rstd[0].double()[:, None])
    err = (g["dweight"].double() - want).abs()
    assert bool((err <= 4 * 2.0 ** -24 * want.abs() + 1e-37).all())
    # dx is whole: the last head's row as a call of its own gives it
    last = drl.dr_layernorm_bwd(x[:, -1:].contiguous(), w[-1:].contiguous(), mean[:, -1:].clone(),
                                rstd[:, -1:].clone(), dy[:, -1:].contiguous())
    assert torch.equal(g["dx"][:, -1:], last["dx"])


@pytest.mark.parametrize("N,H,Dk,Dv", [((1 << 24) + 3, 1, 8, 8), ((1 << 22) + 1, 2, 8, 72)])
def test_step_of_many_small_states(N, H, Dk, Dv):
    """N H ceil(Dv / 64) workgroups of 256 threads: past 2^32 threads.  Every state
    is checked: alpha S + k v^T takes four roundings (alpha's among them), and o a
    sum of Dk products of it."""
    import delta_rule_linear_amd as drl
    announce("step", N, H, Dk, Dv)
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    S, q, k, v = r(N, H, Dk, Dv), r(N, 1, Dk), r(N, 1, Dk), r(N, H, Dv)
    la = -torch.rand(H, generator=gen, device="cuda")
    S0 = S.clone()
    o = drl.dr_linear_attn_step(S, q, k, v, la, decay="head")
    u = 2.0 ** -24
    for a in range(0, N, 1 << 20):   # a part at a time, in float64
        at = slice(a, min(N, a + (1 << 20)))
        old = S0[at].double() * la.double().exp()[None, :, None, None]
        new = k[at].double()[..., None] * v[at].double()[:, :, None]
        want = old + new
        size = old.abs() + new.abs()
        assert bool(((S[at].double() - want).abs() <= 5 * u * size).all())
        qd = q[at].double()[..., None]
        err = (o[at].double() - (want * qd).sum(2)).abs()
        assert bool((err <= (Dk + 6) * u * (size * qd.abs()).sum(2)).all())
