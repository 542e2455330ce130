"""GPU parity of the gated scan (forward, backward, step) against its 64-bit definition."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import ops_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


def make(N, T, D, dtype, seed, cu=None, decay=0.1):
    gen = torch.Generator().manual_seed(seed)
    lead = (1, T) if cu is not None else (N, T)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = {"x": r(*lead, D), "g": -decay * torch.nn.functional.softplus(r(*lead, D)), "dout": r(*lead, D)}
    d = {k: v.to(DT[dtype]).cuda() for k, v in d.items()}
    d["init"], d["dfinal"] = r(N, D).cuda(), r(N, D).cuda()
    d["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    return d


def run_and_check(d, gate, use_init=True):
    init, dfin = (d["init"], d["dfinal"]) if use_init else (None, None)
    out, fin = gdn.gated_scan_fwd(d["x"], d["g"], init_state=init, cu_seqlens=d["cu"], input_gate=gate)
    grads = gdn.gated_scan_bwd(d["x"], d["g"], out, d["dout"], init_state=init, dfinal_state=dfin,
                               cu_seqlens=d["cu"], input_gate=gate)
    ro, rf, bo, bf = ref.scan_fwd(d["x"], d["g"], init, d["cu"], gate)
    ref.check(out, ro, bo, "out")
    ref.check(fin, rf, bf, "final state")
    rg, bg = ref.scan_bwd(d["x"], d["g"], out, d["dout"], init, dfin, d["cu"], gate)
    for got, r, b, name in zip(grads, rg, bg, ("dx", "dg", "dinit")):
        ref.check(got, r, b, name)
    return out, fin, grads


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", [(1, 1, 1), (2, 3, 64), (3, 17, 33), (1, 257, 130), (2, 600, 96), (5, 64, 8),
                                   (1, 1025, 66), (300, 2, 24), (1, 5000, 20), (2, 129, 1000), (1, 9000, 19), (2, 4500, 22),
                                   (1, 3001, 24), (4, 700, 81), (30, 90, 257), (85, 40, 36)])
def test_scan_against_the_definition(N, T, D, dtype, gate):
    run_and_check(make(N, T, D, dtype, seed=N * T + D), gate, use_init=(T % 2 == 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 0, 5, 5, 300], [0, 1, 2, 3], [0, 513, 513], [0, 0, 0, 7], [0, 63, 64, 130, 1400]])
@pytest.mark.parametrize("D", [40, 65])
def test_packed_sequences_empty_ones_among_them(cu, D, dtype):
    run_and_check(make(len(cu) - 1, cu[-1], D, dtype, seed=cu[-1], cu=cu), gate=True)
    run_and_check(make(len(cu) - 1, cu[-1], D, dtype, seed=cu[-1] + 1, cu=cu), gate=False, use_init=False)


def test_sequences_without_tokens_pass_their_state_on():
    s = torch.randn(3, 10).cuda()
    x = torch.empty(3, 0, 10).cuda()
    out, fin = gdn.gated_scan_fwd(x, x, init_state=s)
    assert out.shape == x.shape and torch.equal(fin, s)
    _, fin = gdn.gated_scan_fwd(x, x)
    assert (fin == 0).all()
    dx, dg, di = gdn.gated_scan_bwd(None, x, out, x, dfinal_state=s)
    assert dx.shape == x.shape and torch.equal(di, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_at_their_ends(dtype):
    """g = -inf forgets everything, g = 0 keeps everything; strong decay; growth."""
    d = make(2, 400, 48, dtype, seed=3)
    d["g"][:, 5] = float("-inf")
    d["g"][0, 100:200] = 0.0
    d["g"][1, 300:] = -60.0
    d["g"][:, :, 7] = float("-inf")
    d["g"][:, 20:40, 9] = 0.25
    out, _, _ = run_and_check(d, gate=False)
    assert torch.equal(out[:, :, 7], d["x"][:, :, 7])
    run_and_check(d, gate=True)


def test_growth_out_of_an_exact_zero_stays_zero():
    x = torch.zeros(1, 3000, 32).cuda()
    g = torch.full_like(x, 1.0)
    out, fin = gdn.gated_scan_fwd(x, g)
    assert (out == 0).all() and (fin == 0).all()
    dx, dg, di = gdn.gated_scan_bwd(None, g, out, x)
    assert (dx == 0).all() and (dg == 0).all() and (di == 0).all()


def test_nan_stays_in_its_channel_and_behind_its_token():
    d = make(1, 700, 64, "f32", seed=9)
    clean, _ = gdn.gated_scan_fwd(d["x"], d["g"])
    d["x"][0, 333, 5] = float("nan")
    out, _ = gdn.gated_scan_fwd(d["x"], d["g"])
    bad = torch.isnan(out)
    assert bad[0, 333:, 5].all() and bad.sum() == 700 - 333
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 7), (256, 64), (5, 2048), (2, 1001)])
def test_step_against_the_definition_and_the_forward(N, D, dtype, gate):
    d = make(N, 4, D, dtype, seed=D)
    state = d["init"].clone()
    for t in range(4):
        before = state.clone()
        o = gdn.gated_scan_step(state, d["x"][:, t].contiguous(), d["g"][:, t].contiguous(), input_gate=gate)
        ro, rf, bo, bf = ref.scan_fwd(d["x"][:, t:t + 1], d["g"][:, t:t + 1], before, None, gate)
        ref.check(o, ro[:, 0], bo[:, 0], "step out")
        ref.check(state, rf, bf, "step state")


@pytest.mark.parametrize("gate", [False, True])
def test_gradients_against_differences(gate):
    """Directional derivatives of <dout, out> + <dfinal, final> of the 64-bit definition, by central differences.
    The quotient's own error is O(eps^2) = 1e-8 times third derivatives of order 1 to 100 here; the kernels' fp32
    gradients are within 1e-5 of sums of some thousand terms of order 1."""
    d = make(2, 90, 12, "f32", seed=4, decay=0.3)
    out, _ = gdn.gated_scan_fwd(d["x"], d["g"], init_state=d["init"], input_gate=gate)
    grads = gdn.gated_scan_bwd(d["x"], d["g"], out, d["dout"], init_state=d["init"], dfinal_state=d["dfinal"],
                               input_gate=gate)

    def loss(x, g, s):
        o, f, _, _ = ref.scan_fwd(x, g, s, None, gate)
        return ((o * ref.f64(d["dout"])).sum() + (f * ref.f64(d["dfinal"])).sum()).item()

    base = [ref.f64(d[k]) for k in ("x", "g", "init")]
    gen = torch.Generator().manual_seed(5)
    for i in range(3):
        v = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        at = lambda s: loss(*[b + s * v if j == i else b for j, b in enumerate(base)])  # noqa: E731
        num = (at(1e-4) - at(-1e-4)) / 2e-4
        ana = (ref.f64(grads[i]) * v).sum().item()
        scale = (ref.f64(grads[i]) * v).abs().sum().item()
        assert abs(num - ana) <= 2e-5 * scale, (i, num, ana, scale)


def test_same_bits_twice_and_on_another_stream():
    d = make(3, 1500, 200, "bf16", seed=6)
    a = run_and_check(d, gate=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, fin = gdn.gated_scan_fwd(d["x"], d["g"], init_state=d["init"])
        grads = gdn.gated_scan_bwd(d["x"], d["g"], out, d["dout"], init_state=d["init"], dfinal_state=d["dfinal"])
    s.synchronize()
    assert torch.equal(out, a[0]) and torch.equal(fin, a[1])
    assert all(torch.equal(p, q) for p, q in zip(grads, a[2]))


def test_state_in_place_and_pieces_of_a_sequence():
    """final_state may be init_state's buffer; a sequence in two calls is the sequence in one."""
    d = make(2, 700, 72, "f32", seed=8)
    whole, fin = gdn.gated_scan_fwd(d["x"], d["g"], init_state=d["init"])
    state = d["init"].clone()
    parts = []
    for lo, hi in ((0, 301), (301, 700)):
        o, state = gdn.gated_scan_fwd(d["x"][:, lo:hi].contiguous(), d["g"][:, lo:hi].contiguous(), init_state=state,
                                      final_state=state)
        parts.append(o)
    ro, rf, bo, bf = ref.scan_fwd(d["x"], d["g"], d["init"], None, False)
    ref.check(torch.cat(parts, 1), ro, bo, "two calls")
    ref.check(state, rf, bf, "state of two calls")


def test_pointers_off_the_fast_path():
    """Rows of a size or at an address that no vector access fits."""
    for D, off, dtype in ((64, 1, "bf16"), (64, 3, "bf16"), (63, 0, "bf16"), (66, 2, "bf16"), (64, 1, "f32"),
                          (63, 2, "f32"), (63, 3, "bf16")):
        buf = torch.randn(2 * 100 * D + 8).to(DT[dtype]).cuda()
        x = buf[off:off + 100 * D].view(1, 100, D)
        g = -buf[off + 100 * D:off + 200 * D].abs().view(1, 100, D).mul_(0.1)
        d = {"x": x, "g": g, "dout": x.clone(), "init": torch.randn(1, D).cuda(), "dfinal": torch.randn(1, D).cuda(),
             "cu": None}
        run_and_check(d, gate=True)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last sequence and the last channels are where they should be."""
    N, D = 65541, 32776
    x = torch.full((N, 1, D), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-1, 0, -3:] = 5.0
    g = torch.zeros_like(x)
    out, _ = gdn.gated_scan_fwd(x, g, output_final_state=False)
    assert (out[-1, 0, -3:] == 5).all() and (out[-1, 0, :-3] == 2).all() and (out[0] == 2).all()
    assert out.view(-1)[-D * 3:].float().sum().item() == 3 * 2 * D + 9
    del out
    T = 65541
    x = x.view(1, T, D)
    g.fill_(float("-inf"))
    out, fin = gdn.gated_scan_fwd(x, g.view(1, T, D))
    assert (fin[0, -3:] == 5).all() and (fin[0, :-3] == 2).all() and (out[0, -1, -3:] == 5).all()
