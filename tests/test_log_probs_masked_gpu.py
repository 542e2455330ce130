"""Log probabilities, entropies and their gradient of words that a bias masks by the type's lowest value: logits that are
finite, of no probability, and so far away that their difference from the others times their count leaves fp32."""
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


def spans(V, ranges):
    masked = torch.zeros(V, dtype=torch.bool)
    for a, b in ranges:
        masked[a:b] = True
    return masked


# masked words: a chunk in front, several tiles in front, between ordinary ones, behind them, all but one
CASES = [(1000, [(0, 32)]), (1000, [(0, 64), (300, 640)]), (1000, [(0, 990)]), (1000, [(40, 1000)]), (700, [(0, 7), (600, 700)]),
         (1000, [(0, 517), (518, 1000)]), (9000, [(0, 5000), (6000, 8999)])]


@pytest.mark.parametrize("dtype,low", [("bf16", torch.finfo(torch.bfloat16).min), ("bf16", -1e37), ("bf16", -1e30),
                                       ("f32", torch.finfo(torch.float32).min)])
@pytest.mark.parametrize("V,ranges", CASES)
def test_words_masked_by_the_lowest_value(V, ranges, dtype, low):
    """Results and gradients are those of the words that are left: the masked ones' exponentials are 0, and so is all that
    they are multiplied with.  Their own column of h is 1, that of the other words 0."""
    N, D = (2100 if V > 5000 else 40), 16          # 2100 tokens: the tensor cores' pairs take runs of tiles
    gen = torch.Generator().manual_seed(V + len(ranges))
    h, w = torch.randn(N, D, generator=gen), torch.randn(V, D, generator=gen) / 2
    masked = spans(V, ranges)
    h[:, 0], w[:, 0] = 1, 0
    w[masked] = 0
    w[masked, 0] = low
    left = (~masked).nonzero()[:, 0]
    t = left[torch.randint(0, len(left), (N,), generator=gen)]
    t[::9] = -1
    da, db = torch.randn(N, generator=gen), torch.randn(N, generator=gen)
    h, w, t, da, db = h.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), t.int().cuda(), da.cuda(), db.cuda()
    k = min(5, len(left))
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=k)
    small_w = w[left.cuda()]
    place = torch.full((V,), -1, dtype=torch.int32)
    place[left] = torch.arange(len(left), dtype=torch.int32)
    small_t = torch.where(t >= 0, place.cuda()[t.clamp(min=0).long()], -1)
    want, bound = ref.log_probs_fwd(h, small_w, small_t, k)
    more = (V / 128 + 48) / (len(left) / 128 + 48)    # the sums pass the masked words' zeros too
    for got, r, e, name in zip((logp, H, lse, top), (*want[:3], want[4]), (*bound[:3], bound[3][:, None]),
                               ("logp", "entropy", "lse", "top log probabilities")):
        assert torch.isfinite(got).all(), name
        ref.check(got, r, more * e, name)
    assert not masked[ids[t >= 0].cpu().long()].any()
    dh, dw = gdn.linear_log_probs_bwd(h, w, t, lse, H, da, db)
    want, bound = ref.log_probs_bwd(h, small_w, small_t, lse, H, da, db, low_bits=dtype == "bf16")
    ref.check(dh, want[0], more * bound[0], "dh")
    ref.check(dw[left.cuda()], want[1], bound[1], "dweight")
    assert (dw[masked.cuda()] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_masked_target(dtype):
    """A target among the masked words has its logit's distance as its log probability; the entropy is the others'."""
    low = torch.finfo(DT[dtype]).min
    h = torch.zeros(3, 8, dtype=DT[dtype]).cuda()
    w = torch.zeros(600, 8, dtype=DT[dtype]).cuda()
    h[:, 0], w[:, 0] = 1, low
    w[[70, 400], 0] = 0
    t = torch.tensor([0, 70, 599], dtype=torch.int32).cuda()
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=3)
    ln2 = torch.log(torch.tensor(2.0)).item()
    assert torch.allclose(H, torch.full_like(H, ln2), rtol=1e-6) and torch.allclose(lse, torch.full_like(lse, ln2), rtol=1e-6)
    assert abs(logp[1].item() + ln2) < 1e-6 and (logp[[0, 2]] == low).all()
    assert torch.equal(ids.cpu(), torch.tensor([[70, 400, 0]] * 3, dtype=torch.int32))
