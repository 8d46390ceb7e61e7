"""The decay's gradient on the GPU, within a bound that no wrong one passes
(tests/linattn_gate.py; tests/test_linear_attn_gate_cpu.py shows that for each of
these configurations).  The last ones are segments of more than 1024 tokens, which
the kernel sums in several sweeps."""
import pytest

import linattn_gate as gate
from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


@pytest.fixture(autouse=True)
def _one_thread():
    n = torch.get_num_threads()
    torch.set_num_threads(1)
    yield
    torch.set_num_threads(n)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("case", gate.CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_decay_gradient(case, grad):
    """In either type of the other gradients: the decay's own does not depend on it."""
    import delta_rule_linear_amd as drl
    announce("decay gradient", *case, grad)
    B, H, Hk, L, Dk, Dv, decay = case[:7]
    p = gate.problem(*case)
    # rows that all tokens share stay so on the GPU
    one = lambda t: t[:, :, :1].cuda().expand(t.shape) if case[-1] else t.cuda()  # noqa: E731
    state = lambda t: None if t is None else t.cuda()  # noqa: E731
    g = drl.dr_linear_attn_bwd(one(p["q"]), one(p["k"]), one(p["v"]), p["la"].cuda(), state(p["S0"]), one(p["dO"]),
                               state(p["dS"]), decay=decay, grad_dtype=gate.DT[grad])
    r = gate.reference(p, decay, gate.segment_tokens(B, H, Hk, L, Dk, Dv))
    print("worst", gate.check(g["dlog_alpha"], r, decay))


@pytest.mark.parametrize("case", [c for c in gate.CASES if c[3] == 90], ids=lambda c: c[6])
def test_decay_gradient_against_differences(case):
    import delta_rule_linear_amd as drl
    announce("decay gradient, differences", *case)
    p, decay = gate.problem(*case), case[6]
    a = [p[n].cuda() for n in ("q", "k", "v", "la", "S0", "dO", "dS")]
    g = drl.dr_linear_attn_bwd(*a, decay=decay)
    r = gate.reference(p, decay, gate.segment_tokens(*case[:6]))
    d = torch.randn(p["la"].shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
    gate.check_difference(g["dlog_alpha"], r, decay, d, gate.difference(p, decay, d))
