"""The example with the root-mean-square norm, an entropy in its objective, scoring and 8-bit projections: it runs, its
gradients are those of its parts, and its passes agree."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()


def test_everything_together():
    """Passes of the same model that round at different places: bf16 activations (2^-8 each, some ten in a row) to a few per
    cent; with 8 bits in both operands of five projections of D = 256 terms each (2^-4 / sqrt(3) a value, averaged over the
    terms, so some 5 % a projection's output beside the residual stream that passes them by) within a third."""
    from gated_delta_rule_12_gb300 import train_example
    said = []
    losses, off, off8 = train_example.train(steps=6, batch=3, length=80, vocab=200, report=said.append, norm="rms",
                                            entropy=0.01, score=True, fp8=True)
    assert len(losses) == 6 and all(abs(x) < 20 for x in losses)
    assert off < 0.04 and off8 < 0.33, (off, off8)
    assert any("among the best 5" in line for line in said) and any("8 bits" in line for line in said)
    with pytest.raises(ValueError):
        train_example.train(steps=1, fp8=True)


@pytest.mark.parametrize("norm,entropy", [("rms", 0.0), ("rms", 0.1), ("layer", 0.1)])
def test_gradients_reach_every_parameter(norm, entropy):
    from gated_delta_rule_12_gb300 import train_example
    torch.manual_seed(1)
    model = train_example.Model(100, norm).cuda()
    tokens = torch.randint(0, 100, (2, 70), device="cuda")
    model.loss(tokens, tokens.int(), entropy).backward()
    for name, p in model.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name


def test_norm_and_objective_gradients_against_autograd():
    """A residual block and the objective, with the library's functions and with their formulas in fp64 autograd."""
    from gated_delta_rule_12_gb300.train_example import LinearLogProbs, RmsNorm
    gen = torch.Generator().manual_seed(2)
    x, r, w = torch.randn(40, 64, generator=gen), torch.randn(40, 64, generator=gen), 1 + 0.1 * torch.randn(64, generator=gen)
    head, t = torch.randn(90, 64, generator=gen) / 8, torch.randint(-5, 90, (40,), generator=gen)
    a = [v.cuda().requires_grad_() for v in (x, r, w, head)]
    y, s = RmsNorm.apply(*a[:3])
    logp, H = LinearLogProbs.apply(y, a[3], t.int().cuda())
    (logp.sum() + 0.3 * H.sum() + (s * s).sum()).backward()
    b = [v.double().requires_grad_() for v in (x, r, w, head)]
    s = b[0] + b[1]
    y = s * (s.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * b[2]
    lp = torch.log_softmax(y @ b[3].T, -1)
    kept = t >= 0
    H = -(lp.exp() * lp).sum(-1)
    (lp[kept, t[kept]].sum() + 0.3 * H[kept].sum() + (s * s).sum()).backward()
    for p, q in zip(a, b):
        assert ((p.grad.double().cpu() - q.grad).norm() / q.grad.norm()).item() < 1e-5


def test_a_captured_backward():
    """A training step of the parts captured into a graph and replayed: the bits of an eager one."""
    from gated_delta_rule_12_gb300.train_example import LinearLogProbs, RmsNorm
    gen = torch.Generator().manual_seed(3)
    x, r = (torch.randn(30, 128, generator=gen).to(torch.bfloat16).cuda().requires_grad_() for _ in range(2))
    w, head = torch.ones(128).cuda().requires_grad_(), torch.randn(50, 128, generator=gen).to(torch.bfloat16).cuda().requires_grad_()
    t = torch.arange(30, dtype=torch.int32).cuda()
    leaves = (x, r, w, head)

    def step():
        y, s = RmsNorm.apply(x, r, w)
        logp, H = LinearLogProbs.apply(y, head, t)
        return logp.sum() + H.sum() + s.float().sum()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(step(), leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = torch.autograd.grad(step(), leaves)
    g.replay()
    eager = torch.autograd.grad(step(), leaves)
    assert all(torch.equal(p, q) for p, q in zip(captured, eager))
