"""GPU parity of the linear cross entropy (loss and gradient) against its 64-bit definition."""
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


def make(N, D, V, dtype, seed, ignored=0.1, spread=2.0):
    gen = torch.Generator().manual_seed(seed)
    h = torch.randn((N, D), generator=gen)
    w = torch.randn((V, D), generator=gen) * (spread * D ** -0.5)
    t = torch.randint(0, V, (N,), generator=gen)
    t[torch.rand(N, generator=gen) < ignored] = -100
    dl = torch.rand(N, generator=gen) / N
    return h.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), t.to(torch.int32).cuda(), dl.cuda()


def run_and_check(h, w, t, dl):
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    rv, bd = ref.ce_fwd(h, w, t)
    ref.check(loss, rv[0], bd[0], "loss")
    ref.check(lse, rv[1], bd[1], "lse")
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    rv, bd = ref.ce_bwd(h, w, t, lse, dl, low_bits=h.dtype == torch.bfloat16)
    ref.check(dh, rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")
    for got, r in ((dh, rv[0]), (dw, rv[1])):   # as a whole, the library's tolerance for bfloat16 results
        n = r.norm().item()
        assert (ref.f64(got) - r).norm().item() <= 5e-3 * n + 1e-30
    return (loss, lse), (dh, dw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", [(1, 1, 1), (1, 8, 2), (3, 16, 17), (127, 64, 129), (128, 128, 128), (130, 72, 1000),
                                   (257, 96, 513), (33, 200, 3001), (600, 136, 260), (5, 1024, 777), (300, 61, 400),
                                   (1, 256, 5003), (513, 520, 1031)])
def test_against_the_definition(N, D, V, dtype):
    run_and_check(*make(N, D, V, dtype, seed=N + D + V))


def test_a_vocabulary_in_several_pieces():
    """Enough tokens for the backward pass to take the vocabulary in pieces, the last of them odd."""
    h, w, t, dl = make(5000, 64, 30011, "bf16", seed=1)
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    pick = torch.tensor([0, 1, 255, 256, 2048, 4999])
    rv, bd = ref.ce_fwd(h[pick.cuda()], w, t[pick.cuda()])
    ref.check(loss[pick.cuda()], rv[0], bd[0], "loss")
    rv, bd = ref.ce_bwd(h[pick.cuda()], w, t[pick.cuda()], lse[pick.cuda()], dl[pick.cuda()], low_bits=True)
    ref.check(dh[pick.cuda()], rv[0], bd[0], "dh")
    # dW of a few rows of the vocabulary, on both sides of its 128-column tiles
    hd, keep = ref.f64(h), (t >= 0).cpu()
    for v in (0, 127, 128, 16383, 16384, 30010):
        p = torch.exp(hd @ ref.f64(w[v]) - ref.f64(lse)) - (t.cpu() == v).double()
        G = torch.where(keep, p * ref.f64(dl), 0.0)
        r = G @ hd
        bound = (ref.BF16 + 1e-4) * (G.abs() @ hd.abs()) + ref.BF16 * r.abs()
        assert ((ref.f64(dw[v]) - r).abs() <= bound).all(), v


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ignored_rows_give_and_take_nothing(dtype):
    """Whatever an ignored row's h, lse and dloss hold; targets beyond the vocabulary are ignored like negative ones."""
    h, w, t, dl = make(150, 80, 300, dtype, seed=2, ignored=0.0)
    drop = torch.zeros(150, dtype=torch.bool)
    drop[::7] = True
    drop = drop.cuda()
    t[drop] = torch.where(torch.arange(int(drop.sum()), device="cuda") % 2 == 0, -1, 300).to(torch.int32)
    clean_f, clean_b = run_and_check(h, w, t, dl)
    h[drop], dl[drop] = float("nan"), float("inf")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    assert torch.equal(loss, clean_f[0]) and torch.equal(lse, clean_f[1]) and (loss[drop] == 0).all()
    lse[drop] = float("nan")
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    assert torch.equal(dh, clean_b[0]) and torch.equal(dw, clean_b[1]) and (dh[drop] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_row_ignored_and_no_rows(dtype):
    h, w, t, dl = make(140, 64, 200, dtype, seed=3)
    t.fill_(-100)
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    assert (loss == 0).all() and (dh == 0).all() and (dw == 0).all()
    loss, lse = gdn.linear_cross_entropy_fwd(h[:0], w, t[:0])
    dh, dw = gdn.linear_cross_entropy_bwd(h[:0], w, t[:0], lse, dl[:0])
    assert loss.numel() == 0 and dh.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(dtype):
    """Logits of several hundred: nothing overflows, the softmax is almost a one-hot."""
    h, w, t, dl = make(100, 64, 500, dtype, seed=4, spread=60.0)
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    rv, bd = ref.ce_fwd(h, w, t)
    assert rv[1].abs().max() > 90
    ref.check(loss, rv[0], bd[0], "loss")
    ref.check(lse, rv[1], bd[1], "lse")
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    rv, bd = ref.ce_bwd(h, w, t, lse, dl, low_bits=dtype == "bf16")
    ref.check(dh, rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_and_nan_logits(dtype):
    """A word whose logit is -inf has probability 0 wherever it lies; all words -inf give lse = -inf; NaN spreads over
    its own row only."""
    N, D, V = 6, 8, 400
    h = torch.zeros(N, D)
    h[:, 0], h[:, 1] = 1.0, torch.arange(N) * 0.1
    w = torch.zeros(V, D)
    w[:, 1] = torch.linspace(-1, 1, V)
    w[130:390, 0] = float("-inf")        # whole tiles of it
    h, w = h.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda()
    t = torch.tensor([0, 1, 128, 395, 399, 5], dtype=torch.int32).cuda()
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    l = ref.f64(h)[:, 1:2] * ref.f64(w)[:, 1] + ref.f64(w)[:, 0]
    r = torch.logsumexp(l, -1)
    assert torch.allclose(ref.f64(lse), r, rtol=1e-5, atol=1e-5)
    assert torch.allclose(ref.f64(loss), r - l[torch.arange(N), t.cpu().long()], rtol=1e-5, atol=1e-5)
    w[:, 0] = float("-inf")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    assert (lse == float("-inf")).all() and torch.isnan(loss).all()
    w[:, 0] = 0
    h[2, 3] = float("nan")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    assert torch.isnan(loss).tolist() == [False, False, True, False, False, False]


def test_gradients_against_differences():
    """Directional derivatives of sum_i dloss_i loss_i of the 64-bit definition by central differences."""
    h, w, t, dl = make(40, 24, 150, "f32", seed=5)
    _, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    grads = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    base = [ref.f64(h), ref.f64(w)]
    gen = torch.Generator().manual_seed(6)
    for i in range(2):
        v = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)

        def at(s):
            a = [b + s * v if j == i else b for j, b in enumerate(base)]
            return (ref.ce_fwd(a[0], a[1], t)[0][0] * ref.f64(dl)).sum().item()

        num = (at(1e-4) - at(-1e-4)) / 2e-4
        terms = ref.f64(grads[i]) * v
        assert abs(num - terms.sum().item()) <= 2e-5 * terms.abs().sum().item(), i


def test_same_bits_twice_and_on_another_stream():
    h, w, t, dl = make(700, 256, 2050, "bf16", seed=7)
    f0 = gdn.linear_cross_entropy_fwd(h, w, t)
    g0 = gdn.linear_cross_entropy_bwd(h, w, t, f0[1], dl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f1 = gdn.linear_cross_entropy_fwd(h, w, t)
        g1 = gdn.linear_cross_entropy_bwd(h, w, t, f1[1], dl)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(f0 + g0, f1 + g1))


def test_workspace_left_dirty_by_another_call():
    """A workspace that the caller keeps, filled with NaN patterns or with a larger call's values."""
    ws = torch.full((gdn.linear_cross_entropy_workspace_size(700, 256, 2050, backward=True),), 255, dtype=torch.uint8,
                    device="cuda")
    for N, D, V in ((700, 256, 2050), (65, 40, 333)):
        h, w, t, dl = make(N, D, V, "bf16", seed=8)
        f0 = gdn.linear_cross_entropy_fwd(h, w, t)
        g0 = gdn.linear_cross_entropy_bwd(h, w, t, f0[1], dl)
        ws0 = torch.full((gdn.linear_cross_entropy_workspace_size(N, D, V),), 255, dtype=torch.uint8, device="cuda")
        f1 = gdn.linear_cross_entropy_fwd(h, w, t, workspace=ws0)
        g1 = gdn.linear_cross_entropy_bwd(h, w, t, f1[1], dl, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(f0 + g0, f1 + g1))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 64), ("bf16", 61)])
def test_error_word_reads_clear_after_a_call(dtype, D):
    h, w, t, dl = make(70, D, 300, dtype, seed=9)
    for backward in (False, True):
        ws = torch.full((gdn.linear_cross_entropy_workspace_size(70, D, 300, DT[dtype], backward),), 255,
                        dtype=torch.uint8, device="cuda")
        if backward:
            gdn.linear_cross_entropy_bwd(h, w, t, lse, dl, workspace=ws)
        else:
            _, lse = gdn.linear_cross_entropy_fwd(h, w, t, workspace=ws)
        gdn.check_device_error(ws)
