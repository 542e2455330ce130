"""The example that runs the layer's operators together: it learns, and its token-by-token form is its parallel form."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_example_learns_and_decodes_what_it_learned():
    """The loss starts at log(vocab) and more than halves.  The two passes round their bf16 activations at different
    places (relative 2^-8 each, some ten of them in a row), so they agree to a few per cent at most."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build, train_example
    build.build()
    losses, off = train_example.train(steps=80, batch=8, length=128, vocab=256, report=lambda s: None)
    assert abs(losses[0] - math.log(256)) < 0.7
    assert losses[-1] < 0.5 * losses[0], losses[::10]
    assert off < 0.04


def test_gradients_reach_every_parameter():
    from gated_delta_rule_12_gb300 import train_example
    torch.manual_seed(1)
    model = train_example.Model(100).cuda()
    tokens = torch.randint(0, 100, (2, 70), device="cuda")
    model.loss(tokens, tokens.int()).backward()
    for name, p in model.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name
