"""GPU parity of the root-mean-square norm (forward, 8-bit output, backward) against its 64-bit definition."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import more_ops_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
SHAPES = [(1, 1), (1, 2), (3, 7), (5, 8), (33, 64), (1000, 128), (7, 129), (16, 200), (130, 256), (19, 1001), (64, 1024),
          (9, 2048), (300, 2056), (5, 5120), (4, 8192), (3, 8200), (2, 16384), (2, 20000), (3, 70001), (4099, 24),
          (2500, 40), (90, 22), (70, 254), (40, 1002), (6, 4098), (3, 10002), (3, 15001), (2600, 513), (2600, 768)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


def make(rows, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, res, dy, dr = r(rows, D), r(rows, D) * (1 + r(rows, 1).abs()), r(rows, D), r(rows, D)
    return [t.to(DT[dtype]).cuda() for t in (x, res, dy, dr)] + [(1 + 0.2 * r(D)).cuda()]


def stored(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def check_fwd(x, res, w, eps=EPS):
    y, s, rstd = gdn.rms_norm_fwd(x, w, residual=res, eps=eps)
    assert (s is None) == (res is None)
    t = stored(x, res)
    if s is not None:
        assert torch.equal(s, t)
    rv, bd = ref.rms_fwd(t, w, eps)
    for got, r, e, name in zip((y, rstd), rv, bd, ("out", "rstd")):
        ref.check(got, r, e, name)
    return y, t, rstd


def check_fp8(x, res, w, eps=EPS):
    q, c, s = gdn.rms_norm_fp8(x, w, residual=res, eps=eps)
    t = stored(x, res)
    if s is not None:
        assert torch.equal(s, t)
    (y, _), (e, _) = ref.rms_fwd(t, w, eps)
    R, D = y.shape
    largest = ref.scales(y, 1)
    assert c.shape == largest.shape and q.dtype == torch.float8_e4m3fn
    off = ((ref.f64(c) * 448 - largest.clamp(min=ref.TINY)).abs() / largest.clamp(min=ref.TINY)).max().item()
    assert off <= (0.5 * (D / 32 + 18) + 10) * ref.U
    ref.check_e4m3(q, ref.spread(c, R, D, 1), y, e * 2, "q")
    return q, c, s


def check_bwd(dy, x, rstd, w, dres):
    grads = gdn.rms_norm_bwd(dy, x, rstd, w, dresidual=dres)
    rv, bd = ref.rms_bwd(dy, x, rstd, w, dres)
    for got, r, e, name in zip(grads, rv, bd, ("dx", "dweight")):
        ref.check(got, r, e, name)
    return grads


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_norm_against_the_definition(rows, D, dtype, residual):
    x, res, dy, dr, w = make(rows, D, dtype, seed=rows + D)
    _, t, rstd = check_fwd(x, res if residual else None, w)
    check_bwd(dy, t, rstd, w, dr if residual else None)
    check_fp8(x, res if residual else None, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(40001, 3), (21003, 9), (21003, 57), (11001, 121), (5003, 249), (5003, 254),
                                    (3001, 505), (1501, 1013), (700, 2049), (311, 4093), (309, 8187), (157, 16377),
                                    (3, 16379), (2, 16383)])
def test_rows_that_start_anywhere(rows, D, dtype):
    x, res, dy, dr, w = make(rows, D, dtype, seed=rows + D)
    _, t, rstd = check_fwd(x, res, w)
    check_bwd(dy, t, rstd, w, dr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [509, 512, 20001])
def test_in_place_and_neighbours(D, dtype):
    """residual_out may be the residual or x, out may be x; rows of an odd length share 16 bytes with their neighbours
    without mixing."""
    x, res, dy, dr, w = make(2400 if D < 1000 else 12, D, dtype, seed=9)
    y0, s0, r0 = gdn.rms_norm_fwd(x, w, residual=res)
    q0, c0, _ = gdn.rms_norm_fp8(x, w, residual=res)
    for which in ("residual", "x"):
        a, b = x.clone(), res.clone()
        y, s, _ = gdn.rms_norm_fwd(a, w, residual=b, residual_out=b if which == "residual" else a)
        assert torch.equal(y, y0) and torch.equal(s, s0)
        a, b = x.clone(), res.clone()
        q, c, s = gdn.rms_norm_fp8(a, w, residual=b, residual_out=b if which == "residual" else a)
        assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(c, c0) and torch.equal(s, s0)
    a, b = x.clone(), res.clone()
    y, s, _ = gdn.rms_norm_fwd(a, w, residual=b, out=a, residual_out=b)
    assert y is a and s is b and torch.equal(y, y0) and torch.equal(s, s0)
    dx0, _ = gdn.rms_norm_bwd(dy, s0, r0, w, dresidual=dr)
    x[1::2], dy[1::2] = float("nan"), float("inf")
    y, s, r = gdn.rms_norm_fwd(x, w, residual=res)
    dx, _ = gdn.rms_norm_bwd(dy, s, r, w, dresidual=dr)
    assert torch.equal(y[::2], y0[::2]) and torch.equal(dx[::2], dx0[::2]) and torch.equal(s[::2], s0[::2])
    assert torch.isnan(y[1::2]).all() and torch.isnan(dx[1::2]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(20, 96), (20, 1000), (4, 9000), (4, 17000)])
def test_without_weight(rows, D, dtype):
    x, res, dy, dr, _ = make(rows, D, dtype, seed=1)
    _, t, rstd = check_fwd(x, res, None)
    check_bwd(dy, t, rstd, None, dr)
    check_fp8(x, None, None)


@pytest.mark.parametrize("D", [16, 100, 2048, 18000])
def test_rows_of_zeros(D):
    """rstd is 1 / sqrt(eps); the 8-bit output is zeros with a scale that is not 0.  eps = 0: infinite rstd, NaN rows."""
    x = torch.zeros(6, D).cuda()
    x[3] = 1
    y, _, rstd = gdn.rms_norm_fwd(x, eps=1e-4)
    assert (y[[0, 5]] == 0).all() and torch.allclose(rstd[[0, 5]].cpu(), torch.full((2,), 100.0), rtol=1e-6)
    q, c, _ = gdn.rms_norm_fp8(x, eps=1e-4)
    assert (q[[0, 5]].float() == 0).all() and (c > 0).all() and (q[3].float() == 448).all()
    y, _, rstd = gdn.rms_norm_fwd(x, eps=0.0)
    assert torch.isinf(rstd[0]) and torch.isnan(y[0]).all() and torch.allclose(y[3], torch.ones_like(y[3]), rtol=1e-6)


@pytest.mark.parametrize("D", [64, 2048, 17000])
def test_rows_beyond_fp32_and_nan(D):
    """Squares beyond fp32: rstd is 0 and so is the row; NaN and infinities stay in their rows."""
    x = torch.randn(8, D).cuda()
    x[1] *= 1e25
    x[4, 3], x[6, 5] = float("nan"), float("inf")
    y, _, rstd = gdn.rms_norm_fwd(x)
    assert rstd[1] == 0 and (y[1] == 0).all() and torch.isnan(y[4]).all() and torch.isnan(y[6, 5]) and rstd[6] == 0
    ok = [0, 2, 3, 5, 7]
    assert torch.isfinite(y[ok]).all()
    q, c, _ = gdn.rms_norm_fp8(x)
    assert torch.isnan(q[4].float()).all() and torch.isfinite(q[ok].float()).all() and torch.isnan(q[6, 5].float())
    assert torch.isfinite(c).all() and (c > 0).all()


def test_no_rows():
    x = torch.empty(0, 33).cuda()
    y, s, r = gdn.rms_norm_fwd(x, residual=x)
    assert y.shape == x.shape and s.shape == x.shape and r.numel() == 0
    dx, dw = gdn.rms_norm_bwd(x, x, r)
    assert dx.shape == x.shape and (dw == 0).all()
    q, c, s = gdn.rms_norm_fp8(x)
    assert q.shape == x.shape and c.shape == (0, 1) and s is None


def test_leading_shape():
    x, res, dy, dr, w = make(60, 256, "bf16", seed=4)
    y, s, r = gdn.rms_norm_fwd(x, w, residual=res)
    y3, s3, r3 = gdn.rms_norm_fwd(x.view(3, 20, 256), w, residual=res.view(3, 20, 256))
    assert torch.equal(y3.view(60, 256), y) and r3.shape == (3, 20) and torch.equal(r3.view(-1), r)
    q, c, _ = gdn.rms_norm_fp8(x.view(3, 20, 256), w)
    assert q.shape == (3, 20, 256) and c.shape == (3, 20, 2)
    q1, c1, _ = gdn.rms_norm_fp8(x[7], w)
    assert torch.equal(q1.view(torch.uint8), q[0, 7].view(torch.uint8)) and torch.equal(c1, c[0, 7])


def test_gradients_against_differences():
    """Directional derivatives of <dout, out> + <dresidual, s> of the 64-bit definition by central differences."""
    x, _, dy, dr, w = make(13, 70, "f32", seed=5)
    _, _, r = gdn.rms_norm_fwd(x, w)
    grads = gdn.rms_norm_bwd(dy, x, r, w, dresidual=dr)
    base = [ref.f64(t) for t in (x, w)]
    gen = torch.Generator().manual_seed(6)
    for i in range(2):
        v = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)

        def at(s):
            args = [p + s * v if j == i else p for j, p in enumerate(base)]
            return ((ref.rms_fwd(*args, EPS)[0][0] * ref.f64(dy)).sum() + (args[0] * ref.f64(dr)).sum()).item()

        num = (at(1e-4) - at(-1e-4)) / 2e-4
        terms = ref.f64(grads[i]) * v
        assert abs(num - terms.sum().item()) <= 1e-5 * terms.abs().sum().item(), i


def test_same_bits_twice_and_on_another_stream():
    x, res, dy, dr, w = make(3000, 384, "bf16", seed=7)
    y, t, r = check_fwd(x, res, w)
    g = check_bwd(dy, t, r, w, dr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f1 = gdn.rms_norm_fwd(x, w, residual=res)
        g1 = gdn.rms_norm_bwd(dy, f1[1], f1[2], w, dresidual=dr)
    s.synchronize()
    f2 = gdn.rms_norm_fwd(x, w, residual=res, stream=s)
    q2 = gdn.rms_norm_fp8(x, w, residual=res, stream=s)
    s.synchronize()
    q3 = gdn.rms_norm_fp8(x, w, residual=res)
    assert all(torch.equal(p, q) for p, q in zip((y, t, r, *g), (*f1, *g1)))
    assert all(torch.equal(p, q) for p, q in zip((y, t, r), f2))
    assert torch.equal(q2[0].view(torch.uint8), q3[0].view(torch.uint8)) and torch.equal(q2[1], q3[1])


def test_captured_and_replayed():
    x, res, dy, dr, w = make(700, 1024, "bf16", seed=8)
    rstd = gdn.rms_norm_fwd(x, w)[2]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [*gdn.rms_norm_fwd(x, w, residual=res), *gdn.rms_norm_bwd(dy, x, rstd, w, dresidual=dr),
               *gdn.rms_norm_fp8(x, w, residual=res)[:2]]
    x.copy_(-x)
    res.copy_(-res)
    g.replay()
    want = [*gdn.rms_norm_fwd(x, w, residual=res), *gdn.rms_norm_bwd(dy, x, rstd, w, dresidual=dr),
            *gdn.rms_norm_fp8(x, w, residual=res)[:2]]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_pointers_off_the_fast_path():
    for D, off in ((64, 1), (2048, 3), (1001, 0), (130, 2)):
        buf = torch.randn(80 * D + 8).to(torch.bfloat16).cuda()
        x, dy, res, dr = (buf[off + i * 20 * D:off + (i + 1) * 20 * D].view(20, D) for i in range(4))
        w = torch.randn(D + 1).cuda()[1:]
        _, t, r = check_fwd(x, res, w)
        check_bwd(dy, t, r, w, dr)
        check_bwd(dy, x, r, w, dr)
        check_fp8(x, res, w)
