"""GPU parity of layer norm (forward, backward) against its 64-bit definition."""
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


def make(rows, D, dtype, seed, offset=0.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = r(rows, D) * (1 + r(rows, 1).abs()) + offset
    return (x.to(DT[dtype]).cuda(), (1 + 0.2 * r(D)).cuda(), r(D).cuda(), r(rows, D).to(DT[dtype]).cuda())


def run_and_check(x, w, b, dy, eps=1e-5):
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, eps=eps)
    rv, bd = ref.norm_fwd(x, w, b, eps)
    for got, r, e, name in zip((y, mean, rstd), rv, bd, ("out", "mean", "rstd")):
        ref.check(got, r, e, name)
    grads = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    rv, bd = ref.norm_bwd(dy, x, mean, rstd, w)
    for got, r, e, name in zip(grads, rv, bd, ("dx", "dweight", "dbias")):
        ref.check(got, r, e, name)
    return (y, mean, rstd), grads


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 1), (1, 2), (3, 7), (5, 8), (33, 64), (1000, 128), (7, 129), (16, 200),
                                    (130, 256), (19, 1001), (64, 1024), (9, 2048), (300, 2056), (5, 5120), (4, 8192),
                                    (3, 8200), (2, 20000), (3, 70001), (4099, 24), (2500, 40), (90, 22),
                                    (70, 254), (40, 1002), (6, 4098), (3, 10002), (3, 15001)])
def test_norm_against_the_definition(rows, D, dtype):
    run_and_check(*make(rows, D, dtype, seed=rows + D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(40001, 3), (21003, 9), (21003, 57), (11001, 121), (5003, 249), (5003, 251),
                                    (5003, 254), (3001, 505), (1501, 1013), (700, 2049), (311, 4093), (309, 8187),
                                    (157, 16377), (3, 16379), (2, 16383)])
def test_rows_that_start_anywhere(rows, D, dtype):
    """Several rows a thread where rows start at every place of a 16-byte chunk, and at the edges of the teams."""
    run_and_check(*make(rows, D, dtype, seed=rows + D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_neighbours_in_a_chunk_do_not_mix(dtype):
    """Rows of an odd length share their first and last 16 bytes with other rows; out may be x."""
    x, w, b, dy = make(60, 509, dtype, seed=9)
    y0, m0, r0 = gdn.layer_norm_fwd(x, w, b)
    dx0, _, _ = gdn.layer_norm_bwd(dy, x, m0, r0, w)
    z = x.clone()
    gdn.layer_norm_fwd(z, w, b, out=z)
    assert torch.equal(z, y0)
    x[1::2], dy[1::2] = float("nan"), float("inf")
    y, m, r = gdn.layer_norm_fwd(x, w, b)
    dx, _, _ = gdn.layer_norm_bwd(dy, x, m, r, w)
    assert torch.equal(y[::2], y0[::2]) and torch.equal(dx[::2], dx0[::2])
    assert torch.isnan(y[1::2]).all() and torch.isnan(dx[1::2]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(20, 96), (20, 1000), (4, 9000)])
def test_without_weight_or_bias(rows, D, dtype):
    x, _, b, dy = make(rows, D, dtype, seed=1)
    run_and_check(x, None, None, dy)
    run_and_check(x, None, b, dy)


@pytest.mark.parametrize("D", [64, 1000, 2048, 10000])
def test_rows_far_from_zero(D):
    """A mean of a thousand deviations: a variance from the squares' mean would lose all its bits."""
    run_and_check(*make(12, D, "f32", seed=2, offset=3000.0))


@pytest.mark.parametrize("D", [1, 16, 100, 2048])
def test_constant_rows(D):
    """No variance: out is the bias, rstd is 1 / sqrt(eps)."""
    x = torch.full((6, D), 2.0).cuda()
    w, b = torch.rand(D).cuda() + 0.5, torch.randn(D).cuda()
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, eps=1e-5)
    assert torch.equal(y, b.expand_as(y)) and (mean == 2).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("D", [64, 2048])
def test_rows_whose_variance_leaves_fp32(D):
    """Squares beyond fp32: rstd is 0 and the row its bias, as 1 / sqrt(inf) has it; no NaN."""
    x = torch.randn(3, D).cuda()
    x[1] *= 1e25
    b = torch.randn(D).cuda()
    y, mean, rstd = gdn.layer_norm_fwd(x, None, b)
    assert rstd[1] == 0 and torch.equal(y[1], b) and torch.isfinite(mean).all()
    assert torch.isfinite(y).all() and (rstd[[0, 2]] > 0).all()


def test_rows_do_not_mix():
    """NaN and infinities stay in their rows, and reach the sums over rows."""
    x, w, b, dy = make(40, 512, "f32", seed=3)
    y0, m0, r0 = gdn.layer_norm_fwd(x, w, b)
    dx0, _, _ = gdn.layer_norm_bwd(dy, x, m0, r0, w)
    x[7, 3], x[21, 500] = float("nan"), float("inf")
    y, m, r = gdn.layer_norm_fwd(x, w, b)
    dx, dw, db = gdn.layer_norm_bwd(dy, x, m, r, w)
    ok = torch.ones(40, dtype=torch.bool)
    ok[7] = ok[21] = False
    assert torch.isnan(y[7]).all() and torch.isnan(y[21]).any()
    assert torch.equal(y[ok], y0[ok]) and torch.equal(dx[ok], dx0[ok])
    assert torch.isnan(dw[3]) and torch.isfinite(db).all()


def test_no_rows():
    x = torch.empty(0, 33).cuda()
    y, m, r = gdn.layer_norm_fwd(x)
    assert y.shape == x.shape and m.numel() == 0
    dx, dw, db = gdn.layer_norm_bwd(x, x, m, r)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


def test_leading_shape_and_in_place():
    x, w, b, dy = make(60, 256, "bf16", seed=4)
    y, m, r = gdn.layer_norm_fwd(x, w, b)
    y3, m3, r3 = gdn.layer_norm_fwd(x.view(3, 20, 256), w, b)
    assert torch.equal(y3.view(60, 256), y) and m3.shape == (3, 20) and torch.equal(m3.view(-1), m)
    z = x.clone()
    gdn.layer_norm_fwd(z, w, b, out=z)
    assert torch.equal(z, y)


def test_gradients_against_differences():
    """Directional derivatives of <dout, out> of the 64-bit definition by central differences: an error of 1e-8 of
    the quotient, and of some 1e-6 of the terms' magnitudes for the fp32 gradients."""
    x, w, b, dy = make(13, 70, "f32", seed=5)
    _, m, r = gdn.layer_norm_fwd(x, w, b)
    grads = gdn.layer_norm_bwd(dy, x, m, r, w)
    base = [ref.f64(t) for t in (x, w, b)]
    gen = torch.Generator().manual_seed(6)
    for i in range(3):
        v = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)

        def at(s):
            args = [p + s * v if j == i else p for j, p in enumerate(base)]
            return (ref.norm_fwd(*args, 1e-5)[0][0] * ref.f64(dy)).sum().item()

        num = (at(1e-4) - at(-1e-4)) / 2e-4
        terms = ref.f64(grads[i]) * v
        assert abs(num - terms.sum().item()) <= 1e-5 * terms.abs().sum().item(), i


def test_same_bits_twice_and_on_another_stream():
    x, w, b, dy = make(3000, 384, "bf16", seed=7)
    f0, g0 = run_and_check(x, w, b, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f1 = gdn.layer_norm_fwd(x, w, b)
        g1 = gdn.layer_norm_bwd(dy, x, f1[1], f1[2], w)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(f0 + g0, f1 + g1))


def test_pointers_off_the_fast_path():
    for D, off in ((64, 1), (2048, 3), (1001, 0), (130, 2)):
        buf = torch.randn(40 * D + 8).to(torch.bfloat16).cuda()
        x, dy = buf[off:off + 20 * D].view(20, D), buf[off + 20 * D:off + 40 * D].view(20, D)
        w = torch.randn(D + 1).cuda()[1:]
        run_and_check(x, w, w, dy)


def test_offsets_beyond_32_bits():
    rows, D = 1 << 20, 2056
    x = torch.zeros((rows, D), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(D, device="cuda") % 2 * 2 - 1
    y, m, r = gdn.layer_norm_fwd(x)
    assert torch.equal(y[-1], x[-1]) and (y[-2] == 0).all() and abs(r[-1].item() - 1) < 1e-4
    dx, dw, db = gdn.layer_norm_bwd(x, x, m, r)
    assert (dx[-2] == 0).all() and torch.allclose(dw, torch.ones_like(dw), rtol=1e-4)
    assert torch.equal(db, x[-1].float())
