"""The linear cross entropy at the ends of its sizes: many tokens, many words."""
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
