"""Sizes near the ends of their types, and refusals of the cross entropy's self-test; no GPU is needed."""
import pytest
import torch

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


BIG = 2 ** 32 + 5   # its low 32 bits are 5


def wide(*shape, dtype=torch.float32):
    """A tensor of this shape in one element's memory."""
    return torch.zeros((), dtype=dtype).expand(shape)


@pytest.mark.parametrize("call", [
    lambda: gdn.gated_scan_fwd(wide(1, BIG, 1), wide(1, BIG, 1)),
    lambda: gdn.gated_scan_fwd(wide(1, 1, BIG), wide(1, 1, BIG)),
    lambda: gdn.gated_scan_bwd(None, wide(BIG, 1, 1), wide(BIG, 1, 1), wide(BIG, 1, 1)),
    lambda: gdn.gated_scan_step(wide(BIG, 1), wide(BIG, 1), wide(BIG, 1)),
    lambda: gdn.layer_norm_fwd(wide(1, BIG)),
    lambda: gdn.layer_norm_bwd(wide(1, BIG), wide(1, BIG), wide(1), wide(1)),
    lambda: gdn.linear_cross_entropy_fwd(wide(1, 8), wide(BIG, 8), wide(1, dtype=torch.int32)),
    lambda: gdn.linear_cross_entropy_bwd(wide(BIG, 8), wide(3, 8), wide(BIG, dtype=torch.int32), wide(BIG), wide(BIG)),
])
def test_sizes_beyond_32_bits_are_refused(call):
    with pytest.raises(ValueError, match="2\\^31"):
        call()


def test_workspaces_of_sizes_beyond_32_bits():
    assert gdn.layer_norm_bwd_workspace_size(3, BIG) == 0
    assert gdn.linear_cross_entropy_workspace_size(BIG, 8, 5) == gdn.linear_cross_entropy_workspace_size(4, 8, BIG) == 0


FAKE = 1 << 20
STALL = dict(step=1, limit=1000, h=FAKE, w=FAKE, t=FAKE, lse=FAKE, dl=FAKE, out0=FAKE, out1=FAKE, N=4, D=16, V=32, ws=FAKE,
             wsb=1 << 40, stream=None)


@pytest.mark.parametrize("over,code", [(dict(step=-1), 1), (dict(step=3), 1), (dict(limit=0), 1), (dict(limit=1000001), 1),
                                       (dict(h=None), 1), (dict(lse=None), 1), (dict(dl=FAKE + 2), 1), (dict(out0=None), 1),
                                       (dict(out1=FAKE + 8), 1), (dict(N=0), 1), (dict(D=12), 2), (dict(ws=None), 3),
                                       (dict(wsb=64), 3)])
def test_selftest_refusals(over, code):
    assert gdn.load_library().gdn_selftest_linear_cross_entropy_timeout(*{**STALL, **over}.values()) == code
