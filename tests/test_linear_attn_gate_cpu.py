"""The bound on the decay's gradient (tests/linattn_gate.py) rejects wrong
gradients in every configuration that the GPU runs; the mistakes are made in the
float64 values, on the CPU."""
import pytest

torch = pytest.importorskip("torch")
import linattn_gate as gate  # noqa: E402

SWEEP = 1024   # tokens that the kernel sums at a time


@pytest.fixture(autouse=True)
def _one_thread():
    """Token by token the tensors are small: threads only wait for each other."""
    n = torch.get_num_threads()
    torch.set_num_threads(1)
    yield
    torch.set_num_threads(n)


def wrong(r, decay, strong=False):
    """Named gradients per token with a mistake each.  strong: decays below e^-100,
    whose gradients (but for the few weakest decays') are smaller than the
    rounding of the sums, so that zeros for some of them are no mistake."""
    dla, ends = r["dla"], r["ends"]
    L = dla.shape[-1]
    yield "zero", torch.zeros_like(dla)
    yield "negated", -dla
    if L > 1:
        if not strong:
            first = dla.clone()
            first[:, :, :L // 2] = 0
            yield "first half zero", first
        if decay == "token":
            yield "shifted by a token", torch.roll(dla, 1, -1)
    starts = [0, *ends[:-1]]
    if r["carry"][-1].any():
        last = dla.clone()
        last[:, :, starts[-1]:] -= r["carry"][-1][..., None]
        yield "without <S, dS> at the end", last
    if len(ends) > 1:
        seg = dla.clone()
        for i in range(len(ends) - 1):
            seg[:, :, starts[i]:ends[i]] -= r["carry"][i][..., None]
        yield "without <S, dS> between segments", seg
    if ends[0] > SWEEP:
        # one segment; the later tokens' sum is lost, or counted twice, for all before them
        after = r["terms"][:, :, L - SWEEP:].sum(-1)
        for name, f in (("carry lost", -1), ("carry twice", 1)):
            c = dla.clone()
            c[:, :, :L - SWEEP] += f * after[..., None]
            yield name, c


@pytest.mark.parametrize("case", gate.CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_wrong_gradients_are_rejected(case):
    B, H, Hk, L, Dk, Dv, decay = case[:7]
    p = gate.problem(*case)
    r = gate.reference(p, decay, gate.segment_tokens(B, H, Hk, L, Dk, Dv))
    # the identity that the kernels use gives the direct form's values
    tail = torch.empty_like(r["dla"])
    for i, e in enumerate(r["ends"]):
        s = r["ends"][i - 1] if i else 0
        tail[:, :, s:e] = r["terms"][:, :, s:e].flip(-1).cumsum(-1).flip(-1) + r["carry"][i][..., None]
    assert bool(((tail - r["dla"]).abs() <= 2.0 ** -20 * r["bound"]).all())
    gate.check(gate.total(r["dla"], decay).float(), r, decay)
    for name, x in wrong(r, decay, case[8] < -100):
        with pytest.raises(AssertionError, match="entries off"):
            gate.check(gate.total(x, decay), r, decay)
            pytest.fail(f"{name}: passes")


@pytest.mark.parametrize("case", [c for c in gate.CASES if c[3] == 90], ids=lambda c: c[6])
def test_wrong_gradients_are_off_the_differences(case):
    p, decay = gate.problem(*case), case[6]
    r = gate.reference(p, decay, gate.segment_tokens(*case[:6]))
    d = torch.randn(p["la"].shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
    want = gate.difference(p, decay, d)
    gate.check_difference(gate.total(r["dla"], decay).float(), r, decay, d, want)
    for name, x in wrong(r, decay):
        with pytest.raises(AssertionError, match="off the differences"):
            gate.check_difference(gate.total(x, decay), r, decay, d, want)
            pytest.fail(f"{name}: passes")
