"""Sizes near the ends of their types; no GPU is needed."""
import pytest

import gated_delta_rule_12_gb300 as gdn
from gated_delta_rule_12_gb300 import build as gbuild


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gbuild.build()
    gdn.load_library()


@pytest.mark.parametrize("D", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 64])
def test_workspaces_of_the_longest_rows(D):
    """On the CUDA cores the backward pass keeps a piece's 128 columns of G and dh's sums, one token each here."""
    need = 256 + 128 * 4 + -(-D * 4 // 256) * 256
    assert gdn.linear_cross_entropy_workspace_size(1, D, 2, backward=True) == need
