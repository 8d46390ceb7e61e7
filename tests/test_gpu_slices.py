"""Tensors that start anywhere, on the GPU: slices over rows of odd widths,
statistics and weights of a layer in a packed table, decays of one layer or one
sequence.  Bounds as in tests/test_gpu_layernorm.py and tests/linattn_ref.py."""
import pytest

import linattn_ref as ref
import test_gpu_layernorm as norm
import test_gpu_linear_attn as attn
from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = norm.U


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def check_bwd(t, per_head, mean, rstd, g, out):
    """As test_gpu_layernorm.test_backward: n = (x - mean) rstd is off by 3 u |n|."""
    d = lambda v: v.double().cpu()  # noqa: E731
    dx, dw, db = ref.norm_backward(d(t["x"]), d(t["w"]), d(mean), d(rstd), d(t["dy"]), per_head)
    n = ((d(t["x"]) - d(mean)[..., None]) * d(rstd)[..., None]).abs()
    dy = d(t["dy"]).abs()
    tt = dy * norm.wide(t["w"], per_head).abs()
    D = n.shape[-1]
    bound = d(rstd)[..., None] * U * (8 * tt + (D + 8) * tt.mean(-1, keepdim=True) +
                                      (D + 12) * n * (tt * n).mean(-1, keepdim=True))
    norm.near(g["dx"], dx, bound, "dx", out == "bf16")
    over = (0, 2) if per_head else (0, 1, 2)
    terms = n[..., 0].numel() // (n.shape[1] if per_head else 1)
    norm.near(g["dweight"], dw, (terms + 8) * U * (dy * n).sum(over), "dweight")
    norm.near(g["dbias"], db, (terms + 8) * U * dy.sum(over), "dbias")


@pytest.mark.parametrize("D,dtype,dy_dtype", [(1001, "f32", "f32"), (1001, "bf16", "f32"), (100, "bf16", "bf16"),
                                              (100, "f32", "bf16"), (2, "bf16", "f32"), (1, "f32", "f32"),
                                              (127, "bf16", "bf16"), (4098, "f32", "f32"), (128, "bf16", "bf16"),
                                              (64, "f32", "f32")])
@pytest.mark.parametrize("cut", [1, 2, 3])
def test_norm_of_some_rows(D, dtype, dy_dtype, cut):
    """Rows `cut` on of a [1, 1, L, D] batch, in and out, with what the whole
    batch's forward left as statistics."""
    import delta_rule_linear_amd as drl
    L = 41
    t = norm.data((1, 1, L, D), False, dtype, dy_dtype, "dense", D + cut)
    y, mean, rstd = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"])
    norm.check_fwd(t, False, 1e-5, (y, mean, rstd), dtype)
    part = dict(t, x=t["x"][:, :, cut:], dy=t["dy"][:, :, cut:])
    buf = torch.full_like(t["x"], 9.0)
    out = buf[:, :, cut:]
    got = drl.dr_layernorm_fwd(part["x"], t["w"], t["b"], y=out)
    assert got[0] is out and bool((buf[:, :, :cut] == 9).all())
    norm.check_fwd(part, False, 1e-5, got, dtype)
    m, r = mean[:, :, cut:], rstd[:, :, cut:]
    dbuf = torch.full_like(t["x"], 9.0)
    g = drl.dr_layernorm_bwd(part["x"], t["w"], m, r, part["dy"], dx=dbuf[:, :, cut:])
    assert bool((dbuf[:, :, :cut] == 9).all())
    check_bwd(part, False, m, r, g, dtype)


@pytest.mark.parametrize("H,D,per_head", [(3, 63, True), (1, 1001, False), (5, 3, True), (2, 250, True)])
def test_norm_weights_of_a_packed_table(H, D, per_head):
    """The second layer's weight, bias, and statistics of tables of layers."""
    import delta_rule_linear_amd as drl
    t = norm.data((2, H, 17, D), per_head, "bf16", "bf16", "dense", D)
    shape = (H, D) if per_head else (D,)
    for n in ("w", "b"):
        table = torch.full((3, *shape), float("nan"), device="cuda")
        table[1] = t[n]
        t[n] = table[1]
    stats = torch.full((2, 1 + 2 * H * 17 + 1), 5.0, device="cuda")
    mean, rstd = (s[1:-1].view(2, H, 17) for s in stats)
    got = drl.dr_layernorm_fwd(t["x"], t["w"], t["b"], mean=mean, rstd=rstd)
    norm.check_fwd(t, per_head, 1e-5, got, "bf16")
    assert bool((stats[:, [0, -1]] == 5).all())
    check_bwd(t, per_head, mean, rstd, drl.dr_layernorm_bwd(t["x"], t["w"], mean, rstd, t["dy"]), "bf16")


@pytest.mark.parametrize("decay,L", [("head", 300), ("token", 301), ("token", 1027)])
def test_decays_of_one_layer_or_sequence(decay, L):
    """log alpha as a row of a table, and what a call of its own copy gives, bit for bit."""
    import delta_rule_linear_amd as drl
    announce("decays", decay, L)
    p = attn.problem(1, 3, 3, L, 64, 64, decay, "bf16", grad=True)
    table = torch.full((4, *p["la"].shape), float("nan"), device="cuda")
    table[1] = p["la"]
    q = dict(p, la=table[1])
    assert q["la"].data_ptr() % 16
    for a, b in zip(attn.run_fwd(p, decay), attn.run_fwd(q, decay)):
        assert torch.equal(a, b)
    attn.check_fwd(q, decay)
    g, h = attn.run_bwd(p, decay), attn.run_bwd(q, decay)
    assert all(torch.equal(g[n], h[n]) for n in g)
    if decay == "head":
        S, at = p["S0"].clone(), lambda x: x[:, :, 0].contiguous()
        T = S.clone()
        one = drl.dr_linear_attn_step(S, at(p["q"]), at(p["k"]), at(p["v"]), p["la"], decay=decay)
        two = drl.dr_linear_attn_step(T, at(p["q"]), at(p["k"]), at(p["v"]), q["la"], decay=decay)
        assert torch.equal(one, two) and torch.equal(S, T)
