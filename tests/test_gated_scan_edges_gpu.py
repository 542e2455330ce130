"""The gated scan where runs of rows grow or decay beyond what fp32 holds, and at the ends of its sizes."""
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


# Gates that grow for `run` rows and decay for as many, by turns.  Each is exact in both types.  Over a warp's 16 to 64
# rows, or over the rows that one CTA of a cluster takes at a time, they sum to more than 88.7, fp32's largest exponent.
GROWTH = [(2, 160, 40, 2.0, 80, 1e-37), (3, 60, 33, 6.0, 26, 1e-37), (64, 110, 130, 6.0, 26, -1e-36),
          (1, 9000, 19, 0.125, 1100, 1e-30), (2, 4500, 22, 0.25, 500, -1e-30), (1, 1500, 66, 0.5, 250, 3e-25)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,T,D,step,run,start", GROWTH)
def test_tiny_states_through_growth_that_fp32_cannot_hold_by_itself(N, T, D, step, run, start, dtype):
    """exp of a run's gates leaves fp32, the states before and behind it do not."""
    x = torch.zeros((N, T, D), dtype=DT[dtype], device="cuda")
    up = torch.arange(T, device="cuda") // run % 2 == 0
    g = torch.where(up, step, -step)[None, :, None].expand(N, T, D).to(DT[dtype]).contiguous()
    init = torch.full((N, D), start, device="cuda")
    out, fin = gdn.gated_scan_fwd(x, g, init_state=init)
    ro, rf, bo, bf = ref.scan_fwd(x, g, init, None, False)
    assert 88.8 < step * run and 1e4 < ro.abs().max() < 3e38
    ref.check(out, ro, bo, "out")
    ref.check(fin, rf, bf, "final state")
    # the same from the end: e grows out of dfinal
    g = g.flip(1).contiguous()
    dx, dg, di = gdn.gated_scan_bwd(None, g, x, x, init_state=init, dfinal_state=init)
    (rx, _, ri), (bx, _, bi) = ref.scan_bwd(None, g, x, x, init, init, None, False)
    assert 1e4 < rx.abs().max() < 3e38
    ref.check(dx, rx, bx, "dx")
    ref.check(di, ri, bi, "dinit")


@pytest.mark.parametrize("N,T,D,step", [(2, 600, 48, 0.5), (2, 600, 48, 4.0), (1, 5000, 19, 0.25)])
def test_what_leaves_fp32_is_infinite(N, T, D, step):
    x = torch.zeros(N, T, D).cuda()
    g = torch.full_like(x, step)
    init = torch.ones(N, D).cuda()
    out, fin = gdn.gated_scan_fwd(x, g, init_state=init)
    t = torch.arange(1, T + 1).double() * step
    big, small = t > 88.8, t < 88.6
    assert torch.isposinf(out[:, big.cuda()]).all() and torch.isposinf(fin).all()
    want = t.exp()[small][None, :, None]
    assert ((ref.f64(out[:, small.cuda()]) - want).abs() <= 6 * ref.U * 2 * T * want).all()
    di = gdn.gated_scan_bwd(None, g, x, x, dfinal_state=-init)[2]
    assert torch.isneginf(di).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(700, 40), (9000, 19)])
def test_zero_states_stay_zero_and_new_inputs_decay(T, D, dtype):
    """Rows that grow to beyond fp32 out of nothing, then inputs that decay: no NaN comes of it."""
    x = torch.zeros((1, T, D), dtype=DT[dtype], device="cuda")
    g = torch.full_like(x, 2.0)
    x[:, T // 2:], g[:, T // 2:] = 1.0, -0.5
    out, fin = gdn.gated_scan_fwd(x, g)
    ro, rf, bo, bf = ref.scan_fwd(x, g, None, None, False)
    assert (out[:, :T // 2] == 0).all()
    ref.check(out, ro, bo, "out")
    ref.check(fin, rf, bf, "final state")


def test_the_longest_sequence():
    T = 2 ** 31 - 1
    x = torch.zeros((1, T, 1), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros_like(x)
    x[0, 5], x[0, -1], g[0, 1 << 30] = 3.0, 1.0, float("-inf")
    out, fin = gdn.gated_scan_fwd(x, g)
    assert (out[0, :5] == 0).all() and (out[0, 5:1 << 30] == 3).all() and (out[0, 1 << 30:-1] == 0).all()
    assert out[0, -1] == 1 and fin.item() == 1
    del out
    dfin = torch.full((1, 1), 2.0, device="cuda")
    dx, dg, di = gdn.gated_scan_bwd(None, g, x, torch.zeros_like(x), dfinal_state=dfin)
    assert (dx[0, 1 << 30:] == 2).all() and (dx[0, :1 << 30] == 0).all() and di.item() == 0
    # h_{t-1} is 3 behind token 5 alone, where nothing comes back any more; behind the last token there is none
    assert (dg == 0).all()


def test_the_widest_row():
    D = 2 ** 31 - 1
    x = torch.full((1, 1, D), 2.0, dtype=torch.bfloat16, device="cuda")
    x[0, 0, -3:] = 5.0
    out, fin = gdn.gated_scan_fwd(x, torch.zeros_like(x))
    assert torch.equal(out, x) and (fin[0, -3:] == 5).all() and (fin[0, :-3] == 2).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,gate", [(16, False), (13, True)])
@pytest.mark.parametrize("cu", [[0, 0, 9000, 9007, 9007, 12000], [0, 4001, 4001, 4002, 11000], [0, 8577]])
def test_packed_sequences_in_clusters(cu, D, dtype, gate):
    """Few channels over a long time: the CTAs of a cluster share each sequence, those without a token and those shorter
    than one CTA's rows among them."""
    gen = torch.Generator().manual_seed(cu[-1] + D)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    T, N = cu[-1], len(cu) - 1
    x, dout = r(1, T, D).to(DT[dtype]).cuda(), r(1, T, D).to(DT[dtype]).cuda()
    g = (-0.1 * torch.nn.functional.softplus(r(1, T, D))).to(DT[dtype]).cuda()
    init, dfin = r(N, D).cuda(), r(N, D).cuda()
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    out, fin = gdn.gated_scan_fwd(x, g, init_state=init, cu_seqlens=c, input_gate=gate)
    ro, rf, bo, bf = ref.scan_fwd(x, g, init, c, gate)
    ref.check(out, ro, bo, "out")
    ref.check(fin, rf, bf, "final state")
    grads = gdn.gated_scan_bwd(x, g, out, dout, init_state=init, dfinal_state=dfin, cu_seqlens=c, input_gate=gate)
    rg, bg = ref.scan_bwd(x, g, out, dout, init, dfin, c, gate)
    for got, want, b, name in zip(grads, rg, bg, ("dx", "dg", "dinit")):
        ref.check(got, want, b, name)
