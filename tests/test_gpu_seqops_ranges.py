"""The RMS norm, the short convolution and the gated recurrence at the ends of their
ranges: many columns and few, sequences of many tiles, offsets past 32 bits, the same
bits every time, values that could be taken for something else."""
import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seqops_ref as ref  # noqa: E402
from seqops_ref import d, near  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_rule_linear_amd as drl
    drl.lib()


def gates(gen, shape, decay):
    return -torch.rand(shape, generator=gen) if decay == "log" else 2 + 2 * torch.randn(shape, generator=gen)


# (1100, 300, 8) and (40, 260, 1700): so many columns that a workgroup walks whole sequences; (1, 4500, 130) and
# (2, 2300, 1100): tiles of a column in many workgroups, columns not a multiple of eight
@pytest.mark.parametrize("decay,inputs", [("log", "blend"), ("logit", "unit")])
@pytest.mark.parametrize("B,L,C", [(1100, 300, 8), (40, 260, 1700), (1, 4500, 130), (2, 2300, 1100), (66000, 2, 9)])
def test_scan_walks(B, L, C, decay, inputs):
    import delta_rule_linear_amd as drl
    announce("gated scan", B, L, C, decay, inputs)
    gen = torch.Generator().manual_seed(L)
    x, dh = torch.randn((B, L, C), generator=gen).cuda(), torch.randn((B, L, C), generator=gen).cuda()
    g = gates(gen, (B, L, C), decay).cuda()
    h0, dlast = torch.randn((B, C), generator=gen).cuda(), torch.randn((B, C), generator=gen).cuda()
    m = dict(decay=decay, inputs=inputs)
    h, last = drl.dr_gated_scan_fwd(x, g, h0, **m)
    got = drl.dr_gated_scan_bwd(x, g, h0, h, dh, dlast, **m)
    # three spots of the batch in 64 bits, all channels
    for b in sorted({0, B // 2, B - 1}):
        at = lambda t: d(t[b:b + 1])  # noqa: E731
        want, wlast = ref.scan_forward(at(x), at(g), at(h0), decay, inputs)
        e, elast = ref.scan_errors(at(x), at(g), at(h0), decay, inputs)
        near(h[b:b + 1], want, e, "h")
        near(last[b:b + 1], wlast, elast, "h_final")
        want = ref.scan_backward(at(x), at(g), at(h0), at(h), at(dh), at(dlast), decay, inputs)
        ex, eg, e0 = ref.scan_back_errors(at(x), at(g), want, at(dh), at(dlast), decay, inputs)
        for n, err in (("dx", ex), ("dgate", eg), ("dh0", e0)):
            near(got[n][b:b + 1], want[n], err, n)
    # and every sequence is what it is alone, up to the order in which its tiles are joined
    one, _ = drl.dr_gated_scan_fwd(x[1:2] if B > 1 else x, g[1:2] if B > 1 else g, h0[1:2] if B > 1 else h0, **m)
    k = 1 if B > 1 else 0
    e, _ = ref.scan_errors(d(x[k:k + 1]), d(g[k:k + 1]), d(h0[k:k + 1]), decay, inputs)
    assert ((d(one) - d(h[k:k + 1])).abs() <= 2 * e).all()


def test_the_same_bits_every_time():
    """Tiles of a sequence wait for each other in whatever order they start."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(3)
    x, dh = (torch.randn((2, 7000, 520), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    g = gates(gen, (2, 7000, 520), "logit").to(torch.bfloat16).cuda()
    m = dict(decay="logit", inputs="unit")

    def chain(stream=None):
        h, last = drl.dr_gated_scan_fwd(x, g, None, stream=stream, **m)
        return (h, last) + tuple(drl.dr_gated_scan_bwd(x, g, None, h, dh, stream=stream, **m).values())

    base = chain()
    torch.cuda.synchronize()
    # four at a time, on streams of their own, with workspaces of their own
    for _ in range(5):
        many = [chain(s) for s in [torch.cuda.Stream() for _ in range(4)]]
        torch.cuda.synchronize()
        for got in many:
            assert all(torch.equal(p, q) for p, q in zip(base, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain()
    for _ in range(4):
        graph.replay()
        chain()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, base))
    # a workspace full of anything
    import ctypes
    need = drl._gated_scan_plan(False, (2, 7000, 520, 1, 1, 0, 0, 0, 1, 2), *[(7000 * 520, 0, 520)] * 3, *[(0, 0, 0)] * 3)[2]
    assert need > 0 and ctypes
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        h, last = drl.dr_gated_scan_fwd(x, g, None, workspace=ws, **m)
        assert torch.equal(h, base[0]) and torch.equal(last, base[1])


DECAYS = [("log", g) for g in (0.0, -0.0, -1e-40, -2.0 ** -126, -1e-20, -2.0 ** -24, -0.01, -0.2, -0.39999998, -0.4, -0.40000004,
                               -0.7, -20.0, -87.0, -104.0, -1e30, 1e-20, 0.01)]
DECAYS += [("logit", g) for g in (0.0, -0.0, 0.01, -0.01, 0.5, 1.0, 3.0, 10.0, 20.0, 80.0, -0.5, -3.0, -30.0, -80.0)]


@pytest.mark.parametrize("decay,g", DECAYS)
def test_every_strength_of_decay(decay, g):
    """One decay for 400 tokens, at the borders of its forms, from h0 = 1 without inputs
    and from zero with inputs of one; and its gradients."""
    import delta_rule_linear_amd as drl
    gate = torch.full((1, 400, 8), g, device="cuda")
    for x, h0 in ((torch.zeros((1, 400, 8), device="cuda"), torch.ones((1, 8), device="cuda")),
                  (torch.ones((1, 400, 8), device="cuda"), None)):
        for inputs in ("plain", "blend") + (("unit",) if g <= 0 or decay == "logit" else ()):
            m = dict(decay=decay, inputs=inputs)
            h, _ = drl.dr_gated_scan_fwd(x, gate, h0, **m)
            want, _ = ref.scan_forward(d(x), d(gate), d(h0), decay, inputs)
            e, _ = ref.scan_errors(d(x), d(gate), d(h0), decay, inputs)
            near(h, want, e + 1e-36, "h")   # subnormal products may be lost
            dh = torch.ones_like(h)
            got = drl.dr_gated_scan_bwd(x, gate, h0, h, dh, **m)
            want = ref.scan_backward(d(x), d(gate), d(h0), d(h), d(dh), None, decay, inputs)
            ex, eg, e0 = ref.scan_back_errors(d(x), d(gate), want, d(dh), None, decay, inputs)
            for n, err in (("dx", ex), ("dgate", eg), ("dh0", e0)):
                near(got[n], want[n], err + 1e-36, n)


def test_every_nan_is_passed_on():
    """Maps and states that are NaN of every kind, all bits set among them: what comes
    behind is NaN, and the call ends."""
    import delta_rule_linear_amd as drl
    for bits in (-1, 0x7fc00000, 0x7f800001, -0x400000):
        nan = torch.tensor([bits], dtype=torch.int32).view(torch.float32).cuda()
        x, g = torch.ones((1, 3000, 70), device="cuda"), torch.full((1, 3000, 70), -0.5, device="cuda")
        x[0, 400:1500, 3] = nan
        g[0, 400:1500, 3] = nan
        x[0, 700, 69] = nan
        h, last = drl.dr_gated_scan_fwd(x, g, None, decay="log")
        bad = torch.zeros(h.shape, dtype=torch.bool, device="cuda")
        bad[0, 400:, 3] = bad[0, 700:, 69] = True
        assert torch.equal(torch.isnan(h), bad) and torch.equal(torch.isnan(last[0]), bad[0, -1])
        got = drl.dr_gated_scan_bwd(x, g, None, torch.ones_like(h), torch.ones_like(h), decay="log")
        assert torch.isnan(got["dgate"][0, :1500, 3]).all() and torch.isfinite(got["dgate"][0, 1500:]).all()
        assert torch.isfinite(got["dx"][0, :, :3]).all() and torch.isfinite(got["dx"][0, :, 69]).all()


def test_offsets_past_32_bits():
    """Rows 2^23 elements apart, in a buffer of more than 2^31 bytes: the same as dense."""
    import delta_rule_linear_amd as drl
    gen = torch.Generator().manual_seed(4)
    L, C = 140, 24
    buf = torch.empty((L, 2 ** 23), dtype=torch.float32, device="cuda")       # 4.7 GB
    m = dict(decay="log", inputs="unit")

    def far(t):
        v = buf[:, 5:5 + C][None]
        v.copy_(t)
        return v

    x, dh = torch.randn((1, L, C), generator=gen).cuda(), torch.randn((1, L, C), generator=gen).cuda()
    g = gates(gen, (1, L, C), "log").cuda()
    w = torch.randn((C, 4), generator=gen).cuda()
    h, last = drl.dr_gated_scan_fwd(x, g, None, **m)
    base = drl.dr_gated_scan_bwd(x, g, None, h, dh, **m)
    assert torch.equal(drl.dr_gated_scan_fwd(far(x), g, None, **m)[0], h)
    assert torch.equal(drl.dr_gated_scan_fwd(x, far(g), None, **m)[0], h)
    out = buf[:, 5:5 + C][None]
    drl.dr_gated_scan_fwd(x, g, None, h=out, **m)
    assert torch.equal(out, h)
    for args in ((far(x), g, None, h, dh), (x, far(g), None, h, dh), (x, g, None, far(h), dh), (x, g, None, h, far(dh))):
        if args[0].stride() != x.stride():
            args[0].copy_(x)
        for t, want in zip(args, (x, g, None, h, dh)):   # one of them lies in the buffer
            if t is not None and t.data_ptr() != want.data_ptr():
                t.copy_(want)
        got = drl.dr_gated_scan_bwd(*args, **m)
        assert all(torch.equal(got[n], base[n]) for n in got)
    y, _ = drl.dr_short_conv_fwd(x, w)
    gc = drl.dr_short_conv_bwd(x, w, None, None, dh)
    assert torch.equal(drl.dr_short_conv_fwd(far(x), w)[0], y)
    got = drl.dr_short_conv_bwd(far(x), w, None, None, dh)
    assert all(torch.equal(got[n], gc[n]) for n in got)
    drl.dr_short_conv_fwd(x, w, y=out)
    assert torch.equal(out, y)
    n, rstd, _ = drl.dr_rmsnorm_fwd(x)
    assert torch.equal(drl.dr_rmsnorm_fwd(far(x))[0], n)
    drl.dr_rmsnorm_fwd(x, y=out)
    assert torch.equal(out, n)
    # farther than the recurrence takes
    wide = torch.empty_strided((1, 2, 8), (0, 2 ** 23 + 1, 1), device="cuda")
    with pytest.raises(drl.DeltaRuleError, match="2\\^23"):
        drl.dr_gated_scan_fwd(wide, torch.zeros((1, 2, 8), device="cuda"), decay="log")
    del buf


@pytest.mark.parametrize("B,L,C", [(70000, 1, 9), (1, 1, 70001), (3, 2, 33000)])
def test_wide_and_many(B, L, C):
    import delta_rule_linear_amd as drl
    announce("wide and many", B, L, C)
    gen = torch.Generator().manual_seed(C)
    x = torch.randn((B, L, C), generator=gen).to(torch.bfloat16).cuda()
    w, b = torch.randn((C, 4), generator=gen).cuda(), torch.randn(C, generator=gen).cuda()
    st = torch.randn((B, 3, C), generator=gen).to(torch.bfloat16).cuda()
    y, last = drl.dr_short_conv_fwd(x, w, b, st)
    want = ref.conv_forward(d(x[-1:]), d(w), d(b), d(st[-1:]), True)
    near(y[-1:], want[0], ref.conv_bounds(d(x[-1:]), d(w), d(b), d(st[-1:]), True, want)[1], "y")
    assert torch.equal(d(last[-1:]), want[1])
    g = drl.dr_short_conv_bwd(x, w, b, st, x)
    wg = ref.conv_backward(d(x[-1:]), d(w), d(b), d(st[-1:]), d(x[-1:]), None, True)
    assert float((d(g["dx"][-1:]) - wg["dx"]).norm() / wg["dx"].norm()) < 2.0 ** -7   # bf16, and no more
    if L == 1:
        s2 = st.clone()
        assert torch.equal(drl.dr_short_conv_step(s2, x[:, 0].contiguous(), w, b), y[:, 0]) and torch.equal(s2, last)
