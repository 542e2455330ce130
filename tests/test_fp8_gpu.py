"""GPU parity of the 8-bit quantising and of the product of 8-bit operands against their definitions."""
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


def bits(t):
    return t.view(torch.uint8)


def plain_quantize(x, block_rows):
    """On the CPU in fp32 with IEEE division, as the definition has it."""
    R, D = x.shape
    c = ref.scales(x, block_rows).float().clamp(min=ref.TINY) / 448
    u = x.cpu().float() / ref.spread(c, R, D, block_rows).float()
    return u.clamp(-448, 448).to(torch.float8_e4m3fn), c


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 128), (128, 128), (129, 136), (200, 100), (300, 260), (64, 2048),
                                    (1000, 1001), (2, 20004), (4099, 24), (700, 512), (20000, 128)])
def test_quantize_to_the_bit(rows, D, dtype, block_rows):
    """Scales and values equal the definition's, the many 16-bit values that fall on a border between two steps too."""
    gen = torch.Generator().manual_seed(rows + D)
    x = (torch.randn(rows, D, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen))).to(DT[dtype]).cuda()
    q, c = gdn.fp8_quantize(x, block_rows=block_rows)
    want_q, want_c = plain_quantize(x, block_rows)
    assert q.dtype == torch.float8_e4m3fn and torch.equal(c.cpu(), want_c)
    assert torch.equal(bits(q).cpu(), bits(want_q))


def test_quantize_large_small_zero_and_not_finite():
    x = torch.randn(8, 300).cuda()
    x[0] = 0
    x[1] *= 1e-35
    x[2] *= 1e37
    x[3, 5], x[4, 200] = float("nan"), float("-inf")
    x[5, :] = 3e38
    q, c = gdn.fp8_quantize(x)
    assert (q[0].float() == 0).all() and (c[:4] > 0).all()
    # 2^-100 is the least magnitude a block is scaled to: 1e-35 is some 448 * 1e-35 * 2^100 = 0.006 of its units, of which
    # e4m3 has steps of 2^-9
    assert (c[1] == 2.0 ** -100 / 448).all()
    assert ((ref.f64(q[1].float()) * ref.f64(c[1, 0]) - ref.f64(x[1])).abs() <= 1.01 * 2.0 ** -10 * ref.f64(c[1, 0])).all()
    assert torch.isfinite(c[2]).all() and torch.isnan(q[3, 5].float()) and torch.isfinite(q[3, 6:].float()).all()
    assert torch.isinf(c[4, 1]) and torch.isnan(q[4, 200].float()) and (q[4, 201:256].float() == 0).all()
    assert (q[5].float() == 448).all()
    w, cw = gdn.fp8_quantize(x, block_rows=128)
    assert torch.isfinite(cw[0, 0]) and torch.isinf(cw[0, 1]) and torch.isnan(w[3, 5].float())


def test_quantize_shapes_views_and_streams():
    x = torch.randn(4, 6, 256).cuda()
    q, c = gdn.fp8_quantize(x)
    assert q.shape == x.shape and c.shape == (4, 6, 2)
    flat = torch.randn(20 * 256 + 3).cuda()[3:].view(20, 256)      # off the 16-byte boundaries
    for br in (1, 128):
        want_q, want_c = plain_quantize(flat, br)
        q, c = gdn.fp8_quantize(flat, block_rows=br)
        assert torch.equal(bits(q).cpu(), bits(want_q)) and torch.equal(c.cpu(), want_c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q2, c2 = gdn.fp8_quantize(flat, stream=s)
    s.synchronize()
    q, c = gdn.fp8_quantize(flat)
    assert torch.equal(bits(q), bits(q2)) and torch.equal(c, c2)
    e, ce = gdn.fp8_quantize(torch.empty(0, 200).cuda())
    assert e.shape == (0, 200) and ce.shape == (0, 2)
    e, ce = gdn.fp8_quantize(torch.empty(0, 200).cuda(), block_rows=128)
    assert e.shape == (0, 200) and ce.shape == (0, 2)


def operands(M, N, K, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    w = torch.randn(N, K, generator=gen) * torch.exp(0.5 * torch.randn(N, 1, generator=gen)) * K ** -0.5
    return (*gdn.fp8_quantize(x.cuda()), *gdn.fp8_quantize(w.cuda(), block_rows=128))


def check_linear(M, N, K, seed=0):
    ops = operands(M, N, K, seed)
    out = gdn.fp8_linear(*ops)
    ref.check(out, *ref.fp8_linear(*ops), f"{M} x {N} x {K}")
    return ops, out


@pytest.mark.parametrize("M", [1, 2, 3, 8, 16, 17, 33, 63, 64, 65, 100, 127, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (100, 144), (1000, 640), (257, 16)])
def test_linear_against_the_definition(M, N, K):
    check_linear(M, N, K, seed=M + N + K)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 1, 16), (1, 7, 100), (40, 130, 17), (70, 70, 200), (130, 129, 999),
                                   (64, 2048, 2048), (1, 6144, 2048), (3, 16, 8192), (129, 15, 4112), (700, 1030, 400),
                                   (1025, 515, 1040), (2, 16384, 144), (600, 2000, 2048), (20, 3, 20000), (1000, 3001, 256), (515, 2047, 272)])
def test_linear_odd_and_larger_sizes(M, N, K):
    check_linear(M, N, K, seed=M)


def test_linear_of_no_rows_and_leading_shape():
    x, xs, w, ws = operands(24, 200, 256, seed=1)
    out = gdn.fp8_linear(x, xs, w, ws)
    out3 = gdn.fp8_linear(x.view(4, 6, 256), xs.view(4, 6, 2), w, ws)
    assert out3.shape == (4, 6, 200) and torch.equal(out3.view(24, 200), out)
    one = gdn.fp8_linear(x[5], xs[5], w, ws)
    assert one.shape == (200,)
    assert gdn.fp8_linear(x[:0], xs[:0], w, ws).shape == (0, 200)
    given = torch.empty_like(out)
    assert gdn.fp8_linear(x, xs, w, ws, out=given) is given and torch.equal(given, out)


def test_rows_and_columns_do_not_mix():
    """NaN stays in its row of x and its row of w (a column of out); nothing behind the last row or column is written."""
    x, xs, w, ws = operands(150, 300, 384, seed=2)
    clean = gdn.fp8_linear(x, xs, w, ws)
    xb, wb = bits(x).clone(), bits(w).clone()
    xb[70, 3], wb[200, 300] = 0x7f, 0x7f           # e4m3's NaN
    room = torch.full((152, 300), 7.0, dtype=torch.bfloat16).cuda()
    out = gdn.fp8_linear(xb.view(torch.float8_e4m3fn), xs, wb.view(torch.float8_e4m3fn), ws, out=room[1:151])
    assert (room[0] == 7).all() and (room[151] == 7).all()
    keep = torch.ones(150, 300, dtype=torch.bool).cuda()
    keep[70], keep[:, 200] = False, False
    assert torch.isnan(out[70]).all() and torch.isnan(out[:, 200]).all() and torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("M", [1, 30, 200, 1100])
def test_linear_same_bits_streams_capture_and_workspace(M):
    x, xs, w, ws = operands(M, 640, 1024, seed=3)
    out = gdn.fp8_linear(x, xs, w, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = gdn.fp8_linear(x, xs, w, ws, stream=s)
    s.synchronize()
    size = gdn.fp8_linear_workspace_size(M, 640, 1024)
    room = torch.randint(0, 255, (size,), dtype=torch.uint8).cuda()      # what a workspace holds does not matter
    again = gdn.fp8_linear(x, xs, w, ws, workspace=room)
    gdn.check_device_error(room)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = gdn.fp8_linear(x, xs, w, ws)
    captured.zero_()
    g.replay()
    g.replay()
    assert torch.equal(out, on_s) and torch.equal(out, again) and torch.equal(out, captured)


def test_norm_and_products_in_a_row():
    """The serving path: norm with the residual's addition in 8 bits, projection, quantising, projection back, against the
    same steps in 64 bits on the quantised values."""
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, res, w = r(77, 512).to(torch.bfloat16).cuda(), r(77, 512).to(torch.bfloat16).cuda(), (1 + 0.1 * r(512)).cuda()
    w1, w2 = (gdn.fp8_quantize((r(*s) * s[1] ** -0.5).cuda(), block_rows=128) for s in ((768, 512), (512, 768)))
    q, c, s = gdn.rms_norm_fp8(x, w, residual=res)
    y = gdn.fp8_linear(q, c, *w1)
    ref.check(y, *ref.fp8_linear(q, c, *w1), "projection")
    q2, c2 = gdn.fp8_quantize(y)
    z = gdn.fp8_linear(q2, c2, *w2)
    ref.check(z, *ref.fp8_linear(q2, c2, *w2), "projection back")
    (yr, _), _ = ref.rms_fwd(s, w, 1e-5)
    exact = yr @ (ref.f64(w1[0].float()) * ref.spread(w1[1], 768, 512, 128)).T
    # each value of y is off by 2^-4 of itself at most, 512 of them independent: 3 % of the result's size at most
    assert ((ref.f64(y) - exact).norm() / exact.norm()).item() <= 2.0 ** -4 / 3 ** 0.5 * 1.05
