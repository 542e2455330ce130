"""GPU parity of the token log probabilities, entropies and top alternatives, and of their gradient, against 64 bits."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import more_ops_reference as ref

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
    da, db = torch.randn(N, generator=gen) / N, torch.randn(N, generator=gen) / N
    return h.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), t.to(torch.int32).cuda(), da.cuda(), db.cuda()


def grid(N, D, V, dtype, seed):
    """Values whose products and sums are exact in fp32, so that the logits are, and many of them equal."""
    gen = torch.Generator().manual_seed(seed)
    h = torch.randint(-3, 4, (N, D), generator=gen).float() / 4
    w = torch.randint(-3, 4, (V, D), generator=gen).float() / 8
    t = torch.randint(-2, V, (N,), generator=gen)
    return h.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), t.to(torch.int32).cuda()


def check_fwd(h, w, t, k):
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=k)
    (rp, rH, rl, _, rv), (ep, eH, el, et) = ref.log_probs_fwd(h, w, t, k)
    ref.check(logp, rp, ep, "logp")
    ref.check(H, rH, eH, "entropy")
    ref.check(lse, rl, el, "lse")
    assert (ids is None) == (top is None) == (k == 0)
    if k:
        keep = ((t >= 0) & (t < w.shape[0])).cpu()
        ref.check(top, rv, et[:, None], "top log probabilities")
        assert (ids[~keep.cuda()] == -1).all() and ids.dtype == torch.int32
        i = ids.cpu().long()[keep]
        assert (i >= 0).all() and (i < w.shape[0]).all()
        assert (i.sort(-1).values.diff(dim=-1) > 0).all()          # no word twice
        # the words named are those of the values beside them
        lp = (ref.f64(h).cpu()[keep] @ ref.f64(w).T).gather(1, i) - rl[keep][:, None]
        assert ((lp - ref.f64(top)[keep]).abs() <= et[keep][:, None]).all()
    return logp, H, lse


def check_bwd(h, w, t, lse, H, da, db):
    dh, dw = gdn.linear_log_probs_bwd(h, w, t, lse, H, da, db)
    rv, bd = ref.log_probs_bwd(h, w, t, lse, H, da, db, low_bits=h.dtype == torch.bfloat16)
    ref.check(dh, rv[0], bd[0], "dh")
    ref.check(dw, rv[1], bd[1], "dweight")
    return dh, dw


SIZES = [(1, 1, 1), (1, 8, 2), (3, 16, 17), (127, 64, 129), (128, 128, 128), (130, 72, 1000), (257, 96, 513), (33, 200, 3001),
         (600, 136, 260), (5, 1024, 777), (300, 61, 400), (1, 256, 5003), (513, 520, 1031)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", SIZES)
def test_against_the_definition(N, D, V, dtype):
    h, w, t, da, db = make(N, D, V, dtype, seed=N + D + V)
    k = min(V, (0, 1, 5, 8, 9, 20)[(N + D) % 6])
    logp, H, lse = check_fwd(h, w, t, k)
    check_bwd(h, w, t, lse, H, da, db)
    check_bwd(h, w, t, lse, None, da, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 20])
@pytest.mark.parametrize("N,D,V", [(7, 8, 20), (130, 16, 257), (40, 24, 2000), (3, 40, 9001)])
def test_alternatives_to_the_word(N, D, V, k, dtype):
    """Exact logits, many of them equal: the ids are those of a stable sort."""
    h, w, t = grid(N, D, V, dtype, seed=N + k)
    _, _, _, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=k)
    want = ref.log_probs_fwd(h, w, t, k)[0]
    assert torch.equal(ids.cpu().long(), want[3])
    assert ((ref.f64(top) - want[4]).abs() <= 1e-5 * (1 + want[4].abs())).all()


@pytest.mark.parametrize("k", [5, 20])
def test_alternatives_over_many_tiles(k):
    """Enough tiles that later ones leave out what earlier ones have bettered; columns in rising and in falling order of their
    logits, and all equal."""
    h, w, t = grid(2100, 40, 9000, "bf16", seed=k)
    w[:, 0] = (torch.arange(9000).cuda() // 64 - 70).to(w.dtype)        # rises along the vocabulary
    h[:, 0] = torch.tensor([1.0, -1.0, 0.0]).cuda().repeat(700).to(h.dtype)
    h[5:2100:7, 1:] = 0
    t[::2] = 3
    for _ in range(3):                                                  # what tiles tell one another depends on timing
        _, _, _, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=k)
        l = h.double() @ w.double().T
        v, want = torch.sort(l, dim=-1, descending=True, stable=True)
        keep = ((t >= 0) & (t < 9000))[:, None]
        assert torch.equal(ids.long(), torch.where(keep, want[:, :k], -1))
        lp = torch.where(keep, v[:, :k] - torch.logsumexp(l, -1, keepdim=True), 0.0)
        assert ((top.double() - lp).abs() <= 1e-5 * (1 + lp.abs())).all()


def test_a_vocabulary_in_several_pieces():
    """Enough tokens for the backward pass to take the vocabulary in pieces, the last of them odd."""
    h, w, t, da, db = make(5000, 64, 30011, "bf16", seed=1)
    logp, H, lse, _, _ = gdn.linear_log_probs_fwd(h, w, t, top_k=3)
    dh, dw = gdn.linear_log_probs_bwd(h, w, t, lse, H, da, db)
    pick = torch.tensor([0, 1, 255, 256, 2048, 4999]).cuda()
    rv, bd = ref.log_probs_fwd(h[pick], w, t[pick], 0)
    ref.check(logp[pick], rv[0], bd[0], "logp")
    ref.check(H[pick], rv[1], bd[1], "entropy")
    rv, bd = ref.log_probs_bwd(h[pick], w, t[pick], lse[pick], H[pick], da[pick], db[pick], low_bits=True)
    ref.check(dh[pick], rv[0], bd[0], "dh")
    keep = ((t >= 0) & (t < 30011))[:, None]
    lp = h.double() @ w.double().T - lse.double()[:, None]
    G = -lp.exp() * (da.double()[:, None] + db.double()[:, None] * (lp + H.double()[:, None]))
    G.scatter_add_(1, t.clamp(min=0).long()[:, None], da.double()[:, None])
    r = torch.where(keep, G, 0.0).T @ h.double()
    # two roundings to bf16 of each term, of random signs, and the result's own
    assert ((dw.double() - r).norm() / r.norm()).item() <= 3 * ref.BF16


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_against_differences(dtype):
    """Directional derivatives of <dlogp, logp> + <dentropy, entropy> of the 64-bit definition by central differences."""
    h, w, t, da, db = make(21, 48, 90, dtype, seed=5)
    _, H, lse, _, _ = gdn.linear_log_probs_fwd(h, w, t)
    grads = gdn.linear_log_probs_bwd(h, w, t, lse, H, da, db)
    base = [ref.f64(x) for x in (h, w)]
    bounds = ref.log_probs_bwd(h, w, t, lse, H, da, db, low_bits=dtype == "bf16")[1]
    gen = torch.Generator().manual_seed(6)
    for i in range(2):
        v = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)

        def at(s):
            args = [p + s * v if j == i else p for j, p in enumerate(base)]
            f = ref.log_probs_fwd(*args, t, 0)[0]
            return ((f[0] * ref.f64(da)).sum() + (f[1] * ref.f64(db)).sum()).item()

        num = (at(1e-4) - at(-1e-4)) / 2e-4
        got = ref.f64(grads[i])
        room = ((bounds[i] + (ref.BF16 if dtype == "bf16" else 0.0) * got.abs()) * v.abs()).sum().item()
        assert abs(num - (got * v).sum().item()) <= room + 1e-6 * (got * v).abs().sum().item(), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 61])
def test_same_logp_as_the_cross_entropy(dtype, D):
    """logp is minus the loss, within the roundings of both, and its gradient that of the loss for dloss = -dlogp."""
    h, w, t, da, _ = make(200, D, 700, dtype, seed=3)
    logp, _, lse, _, _ = gdn.linear_log_probs_fwd(h, w, t, top_k=2)
    loss, lse0 = gdn.linear_cross_entropy_fwd(h, w, t)
    assert torch.allclose(logp, -loss, rtol=1e-5, atol=1e-5) and torch.allclose(lse, lse0, rtol=1e-6, atol=1e-6)
    g = gdn.linear_log_probs_bwd(h, w, t, lse0, None, da)
    g0 = gdn.linear_cross_entropy_bwd(h, w, t, lse0, -da)
    assert all(torch.equal(x, y) for x, y in zip(g, g0))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 61), ("f32", 64)])
def test_ignored_rows_and_nan(dtype, D):
    """Ignored rows give zeros and -1 whatever they hold, NaN among it, and reach no gradient; a NaN row that is kept is NaN,
    and alone."""
    h, w, t, da, db = make(300, D, 500, dtype, seed=4)
    t[10:20], t[20], t[30:40] = -100, 500, 7
    clean = gdn.linear_log_probs_fwd(h, w, t, top_k=4)
    g0 = gdn.linear_log_probs_bwd(h, w, t, clean[2], clean[1], da, db)
    h[10:21] = float("nan")
    da[12], db[13] = float("nan"), float("inf")
    out = gdn.linear_log_probs_fwd(h, w, t, top_k=4)
    g = gdn.linear_log_probs_bwd(h, w, t, out[2], out[1], da, db)
    assert all(torch.equal(x, y) for x, y in zip(out, clean)) and all(torch.equal(x, y) for x, y in zip(g, g0))
    assert (out[3][10:21] == -1).all() and all((out[i][10:21] == 0).all() for i in (0, 1, 2, 4)) and (g[0][10:21] == 0).all()
    h[33, 2] = float("nan")
    out = gdn.linear_log_probs_fwd(h, w, t, top_k=4)
    assert all(torch.isnan(out[i][33]).all() for i in (0, 1, 2))
    rest = torch.arange(300) != 33
    assert all(torch.equal(x[rest], y[rest]) for x, y in zip(out, clean))
    t[:] = -100
    out = gdn.linear_log_probs_fwd(h, w, t, top_k=4)
    g = gdn.linear_log_probs_bwd(h, w, t, out[2], out[1], da, db)
    assert all((out[i] == 0).all() for i in (0, 1, 2, 4)) and (out[3] == -1).all() and all((x == 0).all() for x in g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_words_without_a_probability(dtype):
    """Logits of -inf take no part in the entropy and are no alternatives; three words are left of twenty."""
    h = torch.zeros(4, 8, dtype=DT[dtype]).cuda()
    w = torch.zeros(20, 8, dtype=DT[dtype]).cuda()
    h[:, 0], w[:, 0] = 1e20, -3e38
    w[4, 0], w[9, 0], w[17, 0] = 0, 0, 0
    h[:, 1], w[9, 1] = 1, 1
    t = torch.tensor([9, 4, 0, -1], dtype=torch.int32).cuda()
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=5)
    p = torch.softmax(torch.tensor([1.0, 0.0, 0.0], dtype=torch.float64), -1)
    assert torch.equal(ids.cpu(), torch.tensor([[9, 4, 17, -1, -1]] * 3 + [[-1] * 5], dtype=torch.int32))
    assert (top[:3, 3:] == float("-inf")).all() and (top[3] == 0).all()
    assert torch.allclose(top[0, :3].double().cpu(), p.log(), atol=1e-6)
    assert torch.allclose(H[:3].double().cpu(), -(p * p.log()).sum().expand(3), atol=1e-6)
    assert logp[2] == float("-inf") and abs(logp[0].item() - p[0].log().item()) < 1e-6


def test_an_infinite_logit_among_many_tiles():
    """+inf is the best word wherever it stands; its row has no finite results, and the others are as they were."""
    h, w, t, _, _ = make(2100, 64, 9000, "bf16", seed=2, ignored=0.0)
    h[:, 0] = 0
    clean = gdn.linear_log_probs_fwd(h, w, t, top_k=3)
    h[77, 0], w[5003, 0] = 1e20, 3e38
    out = gdn.linear_log_probs_fwd(h, w, t, top_k=3)
    assert out[3][77, 0] == 5003 and not torch.isfinite(out[0][77]) and not torch.isfinite(out[1][77])
    rest = torch.arange(2100) != 77
    assert all(torch.equal(x[rest], y[rest]) for x, y in zip(out, clean))


def test_equal_logits_and_a_sure_word():
    """All words alike: entropy log V and the lowest ids.  One word far above the rest: entropy 0."""
    h, w = torch.zeros(9, 64, dtype=torch.bfloat16).cuda(), torch.randn(1000, 64).to(torch.bfloat16).cuda()
    t = torch.arange(9, dtype=torch.int32).cuda()
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=20)
    lv = torch.log(torch.tensor(1000.0)).item()
    assert (ids == torch.arange(20).cuda()).all() and torch.allclose(H, torch.full_like(H, lv), rtol=1e-6)
    assert torch.allclose(top, torch.full_like(top, -lv), rtol=1e-6) and torch.allclose(logp, -H)
    h[:, 0], w[:, 0], w[321, 0] = 16, 0, 16
    _, H, _, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=1)
    assert (H.abs() < 1e-6).all() and (ids == 321).all() and (top.abs() < 1e-6).all()


def test_no_rows():
    h, w, t = torch.zeros(0, 16).cuda(), torch.zeros(9, 16).cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=3)
    assert logp.shape == (0,) and ids.shape == (0, 3) and top.shape == (0, 3)
    dh, dw = gdn.linear_log_probs_bwd(h, w, t, lse, H, logp, logp)
    assert dh.shape == (0, 16) and (dw == 0).all()


@pytest.mark.parametrize("dtype,N", [("bf16", 100), ("bf16", 3000), ("f32", 100)])
def test_same_bits_streams_capture_and_workspace(dtype, N):
    h, w, t, da, db = make(N, 64, 8000 if N > 1000 else 1500, dtype, seed=8)
    V = w.shape[0]
    out = gdn.linear_log_probs_fwd(h, w, t, top_k=6)
    grads = gdn.linear_log_probs_bwd(h, w, t, out[2], out[1], da, db)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = gdn.linear_log_probs_fwd(h, w, t, top_k=6, stream=s)
    g_s = gdn.linear_log_probs_bwd(h, w, t, out[2], out[1], da, db, stream=s)
    s.synchronize()
    size = max(gdn.linear_log_probs_workspace_size(N, 64, V, 6, DT[dtype]),
               gdn.linear_log_probs_workspace_size(N, 64, V, 6, DT[dtype], backward=True))
    room = torch.randint(0, 255, (size,), dtype=torch.uint8).cuda()      # what a workspace holds does not matter
    again = gdn.linear_log_probs_fwd(h, w, t, top_k=6, workspace=room)
    gdn.check_device_error(room)
    g_again = gdn.linear_log_probs_bwd(h, w, t, out[2], out[1], da, db, workspace=room)
    gdn.check_device_error(room)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = gdn.linear_log_probs_fwd(h, w, t, top_k=6)
        gc = gdn.linear_log_probs_bwd(h, w, t, c[2], c[1], da, db)
    for x in (*c, *gc):
        x.zero_()
    graph.replay()
    graph.replay()
    for got in (on_s + g_s, again + g_again, c + gc):
        assert all(torch.equal(x, y) for x, y in zip(out + grads, got))
