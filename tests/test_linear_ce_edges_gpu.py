"""The linear cross entropy at the ends of its sizes: many tokens, many words in several
pieces, long rows; and what a call leaves whose data never come."""
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


@pytest.mark.parametrize("dtype,D", [("f32", 4), ("bf16", 5)])
def test_more_row_tiles_than_a_grid_has_rows(dtype, D):
    """2^23 tokens, all but some ignored, so that what is left can be taken in 64 bits."""
    N, V = 1 << 23, 100
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn((N, D), generator=gen, device="cuda").to(DT[dtype])
    w = torch.randn((V, D), generator=gen, device="cuda").to(DT[dtype])
    keep = torch.tensor([0, 1, 127, 128, 4 << 20, (4 << 20) + 5, N - 129, N - 128, N - 1], device="cuda")
    t = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    t[keep] = torch.arange(9, device="cuda", dtype=torch.int32) * 11
    dl = torch.rand(N, generator=gen, device="cuda")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    rv, bd = ref.ce_fwd(h[keep], w, t[keep])
    ref.check(loss[keep], rv[0], bd[0], "loss")
    ref.check(lse[keep], rv[1], bd[1], "lse")
    rv, bd = ref.ce_bwd(h[keep], w, t[keep], lse[keep], dl[keep], low_bits=False)
    ref.check(dh[keep], rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")
    other = torch.ones(N, dtype=torch.bool, device="cuda")
    other[keep] = False
    assert (loss[other] == 0).all() and (dh[other] == 0).all()


@pytest.mark.parametrize("dtype,D", [("f32", 4), ("bf16", 3)])
def test_more_word_tiles_than_a_grid_has_rows(dtype, D):
    N, V = 2, 65535 * 128 + 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn((N, D), generator=gen, device="cuda").to(DT[dtype])
    w = torch.randn((V, D), generator=gen, device="cuda").to(DT[dtype])
    t = torch.tensor([7, V - 1], dtype=torch.int32, device="cuda")
    dl = torch.tensor([0.5, 2.0], device="cuda")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    rv, bd = ref.ce_fwd(h, w, t)
    ref.check(loss, rv[0], bd[0], "loss")
    rv, bd = ref.ce_bwd(h, w, t, lse, dl, low_bits=False)
    ref.check(dh, rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")


@pytest.mark.parametrize("D", [1 << 24, (1 << 24) + 8])
def test_very_long_rows(D):
    """The last length of the tensor cores and the first that they leave; sums of a few whole numbers are exact."""
    h = torch.ones((2, D), dtype=torch.bfloat16, device="cuda")
    h[1] = -1
    w = torch.zeros((3, D), dtype=torch.bfloat16, device="cuda")
    w[0, [0, 5, D // 2, D - 1]], w[1, [7, D - 2, D - 1]], w[2, D - 1] = 1.0, 1.0, -1.0
    t = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    l = torch.tensor([[4.0, 3.0, -1.0], [-4.0, -3.0, 1.0]], dtype=torch.float64)
    r = torch.logsumexp(l, -1)
    assert ((ref.f64(lse) - r).abs() <= 1e-6 * (1 + r.abs())).all()
    assert ((ref.f64(loss) - (r - l[[0, 1], [0, 2]])).abs() <= 1e-6 * (1 + r.abs())).all()
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, torch.ones(2, device="cuda"))
    G = torch.softmax(l, -1)
    G[0, 0] -= 1
    G[1, 2] -= 1
    at = torch.tensor([0, 1, 5, 7, D // 2, D - 2, D - 1])
    rh, rw = G @ ref.f64(w[:, at]), G.T @ ref.f64(h[:, at])
    # G in bfloat16 and the result's own rounding; three terms of magnitude 1 at most
    assert ((ref.f64(dh[:, at]) - rh).abs() <= 2 * ref.BF16 * (G.abs() @ ref.f64(w[:, at]).abs())).all()
    assert ((ref.f64(dw[:, at]) - rw).abs() <= 2 * ref.BF16 * (G.abs().T @ ref.f64(h[:, at]).abs())).all()


@pytest.mark.parametrize("step,V,want_dw", [(0, 700, True), (1, 700, True), (1, 3000, True), (2, 700, True), (2, 3000, True),
                                            (2, 3000, False)])
def test_a_wait_that_gives_up_leaves_nan(step, V, want_dw):
    """One tile's loads never come: its waits end at their limit, the error word says so, and what the tile reaches is NaN
    for callers who never read that word; the rest is as always, and so is the next call."""
    N, D = 300, 128
    gen = torch.Generator().manual_seed(step)
    h, w = torch.randn((N, D), generator=gen).bfloat16().cuda(), (torch.randn((V, D), generator=gen) * 0.1).bfloat16().cuda()
    t = torch.randint(0, V, (N,), generator=gen).to(torch.int32).cuda()
    t[10], t[290] = -1, -1
    dl = torch.rand(N, generator=gen).cuda()
    ws = torch.empty(gdn.linear_cross_entropy_workspace_size(N, D, V, backward=step > 0), dtype=torch.uint8, device="cuda")
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    good = (loss, lse) if step == 0 else gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    got = tuple(torch.zeros_like(v) for v in good)
    if not want_dw:
        got = (got[0], None)
    gdn.selftest_linear_cross_entropy_timeout(step, h, w, t, lse, dl, *got, ws, limit_us=50000)
    with pytest.raises(gdn.GDNError) as err:
        gdn.check_device_error(ws)
    assert err.value.code == 5
    # the first tile of 256: rows of the tokens (0 and 1), rows of the words (1 and 2, or tokens again without dweight)
    first = (torch.arange(N) < 256).cuda() & (t >= 0)
    for i, (a, b) in enumerate(zip(got, good)):
        if a is None:
            continue
        if step == 2 and i == 0 and want_dw:
            lost = torch.zeros(N, dtype=torch.bool, device="cuda")
        elif step > 0 and i == 1:
            lost = (torch.arange(V) < 256).cuda()
        else:
            lost = first
        assert torch.isnan(a[lost]).all() and torch.equal(a[~lost], b[~lost]), (step, i)
    again = gdn.linear_cross_entropy_fwd(h, w, t, workspace=ws) if step == 0 else \
        gdn.linear_cross_entropy_bwd(h, w, t, lse, dl, workspace=ws)
    gdn.check_device_error(ws)
    assert all(torch.equal(a, b) for a, b in zip(again, good))


@pytest.mark.parametrize("dtype,D", [("f32", 20), ("bf16", 61), ("bf16", 64)])
def test_several_pieces_of_the_vocabulary(dtype, D):
    """More tokens times words than one piece of the backward pass takes, the last piece partial and odd."""
    N, V = (700, 30011) if (dtype, D) != ("bf16", 64) else (3000, 23001)
    gen = torch.Generator().manual_seed(3)
    h = torch.randn((N, D), generator=gen).to(DT[dtype]).cuda()
    w = (torch.randn((V, D), generator=gen) * (2 * D ** -0.5)).to(DT[dtype]).cuda()
    t = torch.randint(-V // 10, V, (N,), generator=gen).to(torch.int32).cuda()
    t[:4] = torch.tensor([0, V - 1, V, -1])
    dl = (torch.rand(N, generator=gen) / N).cuda()
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    rv, bd = ref.ce_fwd(h, w, t)
    ref.check(loss, rv[0], bd[0], "loss")
    ref.check(lse, rv[1], bd[1], "lse")
    rv, bd = ref.ce_bwd(h, w, t, lse, dl, low_bits=dtype == "bf16" and D == 64)
    ref.check(dh, rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")


@pytest.mark.parametrize("N", [8193, 16700])
def test_more_tokens_than_a_group_of_row_tiles(N):
    """Beyond 8192 tokens the tensor cores' row tiles come in several groups, the last one smaller."""
    D, V = 24, 700
    gen = torch.Generator().manual_seed(N)
    h = torch.randn((N, D), generator=gen).bfloat16().cuda()
    w = (torch.randn((V, D), generator=gen) * (2 * D ** -0.5)).bfloat16().cuda()
    t = torch.randint(-V // 10, V, (N,), generator=gen).to(torch.int32).cuda()
    dl = (torch.rand(N, generator=gen) / N).cuda()
    loss, lse = gdn.linear_cross_entropy_fwd(h, w, t)
    dh, dw = gdn.linear_cross_entropy_bwd(h, w, t, lse, dl)
    rv, bd = ref.ce_fwd(h, w, t)
    ref.check(loss, rv[0], bd[0], "loss")
    ref.check(lse, rv[1], bd[1], "lse")
    rv, bd = ref.ce_bwd(h, w, t, lse, dl, low_bits=True)
    ref.check(dh, rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")
