"""Branches that only large or lopsided calls reach: scales that do not fit the few-token product's table at once, and
alternatives of rows with fewer ordinary words than are asked for, over tiles enough that they tell one another."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import more_ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


@pytest.mark.parametrize("M,N,K", [(100, 130, 40000), (128, 20, 20480), (50, 100, 70000), (40, 40, 140000), (20, 17, 300000),
                                   (3, 9, 300000), (1, 128, 1 << 20), (600, 300, 33000), (7, 5, 30001)])
def test_products_over_a_long_k(M, N, K):
    gen = torch.Generator().manual_seed(K)
    x = gdn.fp8_quantize((torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))).cuda())
    w = gdn.fp8_quantize((torch.randn(N, K, generator=gen) * K ** -0.5).cuda(), block_rows=128)
    # scales of very different size along K, so that one in the wrong place shows
    for c in (x[1], w[1]):
        c *= torch.exp2(torch.randint(-3, 4, (c.shape[1],), generator=gen).float()).cuda()
    ref.check(gdn.fp8_linear(*x, *w), *ref.fp8_linear(*x, *w), "out")


@pytest.mark.parametrize("k", [1, 5, 8, 20])
@pytest.mark.parametrize("left", [0, 1, 4, 30])
@pytest.mark.parametrize("N,D,V,dtype", [(2100, 16, 9000, torch.bfloat16), (8500, 8, 6011, torch.bfloat16), (300, 16, 777, torch.bfloat16),
                                         (300, 16, 777, torch.float32), (130, 9, 500, torch.bfloat16)])
def test_alternatives_where_few_words_are_left(N, D, V, dtype, left, k):
    """Half of the rows: all words but `left` masked by the lowest number, equal to one another, so that the lower indexes follow
    the words that are left.  The other half: by -inf, which is no alternative, so that -1 follows."""
    gen = torch.Generator().manual_seed(N + left)
    low = torch.finfo(dtype).min
    h, w = torch.zeros(N, D), torch.zeros(V, D)
    h[:, 0] = 1
    h[1::2, 0] = 2.0 ** 40                              # times the lowest number: -inf
    w[:, 0] = low
    words = torch.randperm(V, generator=gen)[:left].sort().values
    w[words, 0] = 0
    w[words, 1] = torch.randint(-2, 3, (left,), generator=gen).float()
    h[:, 1] = torch.randint(-2, 3, (N,), generator=gen).float()
    t = torch.randint(-1, V, (N,), generator=gen)
    h, w, t = h.to(dtype).cuda(), w.to(dtype).cuda(), t.int().cuda()
    room = torch.randint(0, 255, (gdn.linear_log_probs_workspace_size(N, D, V, k, dtype),), dtype=torch.uint8).cuda()
    _, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=k, workspace=room)
    l = (h.double() @ w.double().T).float()             # exact, or beyond fp32
    v, want = torch.sort(l, dim=-1, descending=True, stable=True)
    want = torch.where(v > float("-inf"), want, -1)[:, :k]
    keep = (t >= 0)[:, None]
    assert torch.equal(ids.long(), torch.where(keep, want, -1))
    if left:
        lp = torch.log_softmax(l.double(), -1)
        goal = torch.where(want >= 0, lp.gather(1, want.clamp(min=0)), float("-inf"))
        # an exact logit less lse: the sum of `left` exponentials and a few roundings; the lowest number swallows lse
        got, goal = top[keep[:, 0]].double(), goal[keep[:, 0]]
        far = goal < -1e30
        assert (got[far] <= float(low)).all() and ((got - goal).abs() <= 1e-5 * (1 + goal.abs()))[~far].all()
        p = lp.exp()
        rH = -(p * lp.clamp(min=-1e4)).sum(-1)
        assert ((H.double() - rH).abs() <= 1e-5 * (1 + rH))[keep[:, 0]].all()
