"""Layer norm where its buffers alias, its rows are constant or very long."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


def bwd_into(dx, dy, x, mean, rstd, w):
    """The C entry with the caller's dx; returns the weight's and bias's gradients."""
    rows, D = x.shape
    dt = gdn.GDN_BF16 if x.dtype == torch.bfloat16 else gdn.GDN_F32
    dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(gdn.layer_norm_bwd_workspace_size(rows, D, x.dtype), dtype=torch.uint8, device="cuda")
    rc = gdn.load_library().gdn_layer_norm_bwd(dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                               w.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows, D, dt,
                                               ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == gdn.GDN_OK
    return dw, db


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(60, 509), (40, 2048), (9, 9000), (70, 20000)])
def test_dx_in_the_place_of_dout(rows, D, dtype):
    """The same bits as with a dx of its own, for rows in registers and for longer ones."""
    gen = torch.Generator().manual_seed(D)
    x, dy = (torch.randn((rows, D), generator=gen).to(DT[dtype]).cuda() for _ in range(2))
    w = torch.rand(D, generator=gen).cuda() + 0.5
    _, mean, rstd = gdn.layer_norm_fwd(x, w)
    want = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    buf = dy.clone()
    dw, db = bwd_into(buf, buf, x, mean, rstd, w)
    assert torch.equal(buf, want[0])
    assert torch.equal(dw, want[1]) and torch.equal(db, want[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [13, 49, 98, 255, 509, 1000, 1501, 2049, 3001, 7001, 10000, 16383, 20000])
@pytest.mark.parametrize("value", [3.0, 1000.0])
def test_constant_rows_of_any_length(value, D, dtype):
    """Partial sums of whole numbers below 2^24 are exact, so the mean is the value itself, no deviation is left and the
    row becomes its bias, of however many elements it consists."""
    x = torch.full((5, D), value, dtype=DT[dtype]).cuda()
    b = torch.randn(D).cuda()
    y, mean, rstd = gdn.layer_norm_fwd(x, None, b, eps=1e-5)
    assert (mean == value).all()
    assert torch.equal(y, b.to(DT[dtype]).expand_as(y))


def test_the_longest_row():
    """2^31 - 1 elements of +-1: a thread's sums are whole numbers up to 2^23, and the mean is 2^-31."""
    D = 2 ** 31 - 1
    x = torch.ones((1, D), dtype=torch.bfloat16, device="cuda")
    x[0, 1::2] = -1
    y, mean, rstd = gdn.layer_norm_fwd(x)
    assert torch.equal(y, x) and abs(mean.item()) < 1e-6 and abs(rstd.item() - (1 + 1e-5) ** -0.5) < 1e-6
