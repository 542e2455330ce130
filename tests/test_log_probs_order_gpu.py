"""Log probabilities of more tokens than one group of row tiles has, over several windows of words, with a last group of one or
two row tiles: every row's results and alternatives."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import more_ops_reference as ref
from test_log_probs_gpu import grid

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


# tokens, words, alternatives: two groups, the second of one token, one row tile, two; three groups; groups of more than 32 row
# tiles over few words; a second group in several windows itself
SIZES = [(8193, 5000, 20), (8448, 4700, 5), (8500, 6011, 8), (16900, 5377, 3), (80000, 300, 20), (156000, 17, 9),
         (12000, 30011, 5), (8193, 5000, 0)]


@pytest.mark.parametrize("N,V,k", SIZES)
def test_groups_and_windows(N, V, k):
    """Exact logits: ids to the word, each row's numbers within their bounds.  The last rows point at the first and the last words."""
    D = 8
    h, w, t = grid(N, D, V, "bf16", seed=N + V)
    t[-1], t[-2 if N > 1 else -1], t[0] = V - 1, 0, V // 2
    room = torch.full((gdn.linear_log_probs_workspace_size(N, D, V, k) + 256,), 0xff, dtype=torch.uint8, device="cuda")
    logp, H, lse, ids, top = gdn.linear_log_probs_fwd(h, w, t, top_k=k, workspace=room[:-256])
    gdn.check_device_error(room)
    assert (room[-256:] == 0xff).all()
    for i in range(0, N, 4096):
        r = slice(i, min(N, i + 4096))
        if i and r.stop < N - 4096 and i // 4096 % 4:      # a quarter of the middle, and both ends
            continue
        l = h[r].double() @ w.double().T
        keep = (t[r] >= 0) & (t[r] < V)
        m = l.max(-1, keepdim=True).values
        e, d = torch.exp(l - m), l - m
        S = e.sum(-1, keepdim=True)
        lsum = torch.log(S)
        p, rl = e / S, (m + lsum)[:, 0]
        rH = (lsum - (p * d).sum(-1, keepdim=True))[:, 0]
        # the logits are exact; the sums' and exponentials' roundings as the reference of one group counts them
        term = (V / 128 + 48) * ref.U + 6 * ref.U * d.abs()
        eH = (p * term * (1 + d.abs() + (p * d).sum(-1, keepdim=True).abs())).sum(-1) + 6 * ref.U * (rH + lsum[:, 0].abs())
        el = (V / 128 + 40) * ref.U + 4 * ref.U * (rl.abs() + l.abs().max(-1).values)
        at = l.gather(1, t[r].clamp(0, V - 1).long()[:, None])[:, 0] - rl
        for got, want, err, name in ((logp, at, 2 * el, "logp"), (H, rH, eH, "entropy"), (lse, rl, el, "lse")):
            want = torch.where(keep, want, 0.0)
            assert ((got[r].double() - want).abs() <= err).all(), (name, i)
        if k:
            v, word = torch.sort(l, dim=-1, descending=True, stable=True)
            assert torch.equal(ids[r].long(), torch.where(keep[:, None], word[:, :k], -1)), i
            want = torch.where(keep[:, None], v[:, :k] - rl[:, None], 0.0)
            assert ((top[r].double() - want).abs() <= 2 * el[:, None]).all(), i


def test_the_last_group_does_not_change_the_others():
    """The same rows with one token more: the rows of the first group have the same parts, and so the same bits."""
    N, D, V = 8192, 16, 5000
    h, w, t = grid(N + 1, D, V, "bf16", seed=2)
    a = gdn.linear_log_probs_fwd(h[:N].contiguous(), w, t[:N].contiguous(), top_k=7)
    b = gdn.linear_log_probs_fwd(h, w, t, top_k=7)
    assert all(torch.equal(x, y[:N]) for x, y in zip(a, b))
