"""The root-mean-square norm, the 8-bit quantising and product and the log probabilities at their edges: named streams, memory
in use elsewhere, tensors that start anywhere, a wait that gives up, several products at once."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import more_ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


def same(a, b):
    a, b = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v for v in (a, b))
    return torch.equal(a, b)


def operators():
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, res, dy = (r(700, 256).bfloat16() for _ in range(3))
    w, head = r(256), (r(1000, 256) * 0.1).bfloat16()
    t = torch.arange(700, device="cuda", dtype=torch.int32) - 100
    da, db = r(700), r(700)
    _, s, rstd = gdn.rms_norm_fwd(x, w, residual=res)
    q, c = gdn.fp8_quantize(x)
    w8 = gdn.fp8_quantize(head, block_rows=128)
    _, H, lse, _, _ = gdn.linear_log_probs_fwd(x, head, t)
    return {
        "norm": lambda st: gdn.rms_norm_fwd(x, w, residual=res, stream=st),
        "norm in 8 bits": lambda st: gdn.rms_norm_fp8(x, w, residual=res, stream=st),
        "norm backward": lambda st: gdn.rms_norm_bwd(dy, s, rstd, w, dresidual=res, stream=st),
        "quantising": lambda st: gdn.fp8_quantize(x, stream=st),
        "weights": lambda st: gdn.fp8_quantize(head, block_rows=128, stream=st),
        "product": lambda st: (gdn.fp8_linear(q, c, *w8, stream=st),),
        "product of few": lambda st: (gdn.fp8_linear(q[:9], c[:9], *w8, stream=st),),
        "log probabilities": lambda st: gdn.linear_log_probs_fwd(x, head, t, top_k=4, stream=st),
        "gradient": lambda st: gdn.linear_log_probs_bwd(x, head, t, lse, H, da, db, stream=st),
    }


NAMES = ["norm", "norm in 8 bits", "norm backward", "quantising", "weights", "product", "product of few",
         "log probabilities", "gradient"]


@pytest.mark.parametrize("name", NAMES)
def test_named_streams_and_memory_still_in_use(name):
    """The same bits on a named stream, a torch stream or a raw handle, while the current one still uses memory that it has
    given back."""
    call = operators()[name]
    want = call(None)
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        b = a
        for _ in range(20):      # some 10 ms of work in front of the temporaries' use
            b = a @ b
        temps = [torch.empty_like(v) for v in want for _ in range(3)]
        for v in temps:
            v.view(torch.uint8).fill_(7)
        copies = [v.clone() for v in temps]
        del temps, v             # their memory is free, their use is not over
        got = call(stream)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(got, want))
        assert all((c.view(torch.uint8) == 7).all() for c in copies)


@pytest.mark.parametrize("M,N,K", [(3000, 8, 128), (3000, 40, 512), (5000, 136, 64), (4097, 1, 16), (257, 65, 4096),
                                   (1, 16384, 16), (17, 129, 2064)])
def test_products_of_unusual_shapes(M, N, K):
    gen = torch.Generator().manual_seed(M)
    x = gdn.fp8_quantize(torch.randn(M, K, generator=gen).cuda())
    w = gdn.fp8_quantize(torch.randn(N, K, generator=gen).cuda(), block_rows=128)
    ref.check(gdn.fp8_linear(*x, *w), *ref.fp8_linear(*x, *w), "out")


@pytest.mark.parametrize("off", [1, 8, 16])
def test_products_of_tensors_that_start_anywhere(off):
    gen = torch.Generator().manual_seed(off)
    x, xs = gdn.fp8_quantize(torch.randn(50, 256, generator=gen).cuda())
    w, ws = gdn.fp8_quantize(torch.randn(70, 256, generator=gen).cuda(), block_rows=128)
    want = gdn.fp8_linear(x, xs, w, ws)

    def moved(t, n):
        room = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        room[n:].view(torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype).copy_(
            t.reshape(-1).view(torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype))
        return room[n:].view(t.shape)

    bound = ref.fp8_linear(x, xs, w, ws)
    for got in (gdn.fp8_linear(moved(x, off), moved(xs, off), w, ws), gdn.fp8_linear(x, xs, moved(w, off), moved(ws, 1)),
                gdn.fp8_linear(x, xs, w, ws, out=moved(torch.empty_like(want), off))):
        ref.check(got, *bound, "out")


@pytest.mark.parametrize("M,N,K", [(5, 300, 4096), (100, 640, 1024), (2000, 3000, 512)])
def test_a_wait_that_gives_up(M, N, K):
    """One tile's data never comes: nothing faults or hangs, the error word says so, and the tile's results are NaN.  The next
    call is right."""
    gen = torch.Generator().manual_seed(M)
    x = gdn.fp8_quantize(torch.randn(M, K, generator=gen).cuda())
    w = gdn.fp8_quantize(torch.randn(N, K, generator=gen).cuda(), block_rows=128)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    room = torch.empty(gdn.fp8_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    gdn.selftest_fp8_linear_timeout(*x, *w, out, room, limit_us=3000)
    with pytest.raises(gdn.GDNError, match="TIMEOUT"):
        gdn.check_device_error(room)
    assert torch.isnan(out[0, 0]) and torch.isnan(out[min(M, 16) - 1, 127])
    ref.check(gdn.fp8_linear(*x, *w, out=out, workspace=room), *ref.fp8_linear(*x, *w), "out")
    gdn.check_device_error(room)


@pytest.mark.parametrize("N,V,k", [(100, 700, 0), (100, 700, 4), (2600, 9000, 9)])
def test_log_probabilities_whose_wait_gives_up(N, V, k):
    """The same of the log probabilities: the rows of the first pair's tiles are NaN, and the next call is right."""
    gen = torch.Generator().manual_seed(N)
    h, w = torch.randn(N, 64, generator=gen).bfloat16().cuda(), (torch.randn(V, 64, generator=gen) / 4).bfloat16().cuda()
    t = torch.randint(0, V, (N,), generator=gen).int().cuda()
    want = gdn.linear_log_probs_fwd(h, w, t, top_k=k)
    logp, H = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    ids = torch.zeros(N, k, dtype=torch.int32, device="cuda") if k else None
    top = torch.zeros(N, k, device="cuda") if k else None
    room = torch.empty(gdn.linear_log_probs_workspace_size(N, 64, V, k), dtype=torch.uint8, device="cuda")
    gdn.selftest_linear_log_probs_timeout(h, w, t, logp, H, ids, top, room, limit_us=3000)
    with pytest.raises(gdn.GDNError, match="TIMEOUT"):
        gdn.check_device_error(room)
    assert torch.isnan(logp[:100]).all() and torch.isnan(H[:100]).all()
    got = gdn.linear_log_probs_fwd(h, w, t, top_k=k, workspace=room)
    gdn.check_device_error(room)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))


def test_products_at_once():
    """Two streams with products of both kernels and log probabilities next to one another, time and again."""
    ops = operators()
    names = ["product", "product of few", "log probabilities", "norm in 8 bits"]
    want = {n: ops[n](None) for n in names}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):
        n = names[i % len(names)]
        got.append((n, ops[n](streams[i % 3])))
    torch.cuda.synchronize()
    for n, g in got:
        assert all(same(p, q) for p, q in zip(g, want[n])), n


def test_captured_graphs_in_turn():
    """Each operator captured by itself, the graphs replayed in turn on the same inputs: the same bits as eager calls."""
    ops = operators()
    want = {n: ops[n](None) for n in NAMES}
    graphs = {}
    torch.cuda.synchronize()
    for n in NAMES:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs[n] = (g, ops[n](None))
    for _ in range(2):
        for n in reversed(NAMES):
            graphs[n][0].replay()
    for n in NAMES:
        assert all(same(p, q) for p, q in zip(graphs[n][1], want[n])), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", [(40001, 3), (21003, 57), (11001, 121), (5003, 249), (10001, 505), (1501, 1013),
                                    (700, 2049), (311, 4093), (9001, 1024), (40000, 128)])
def test_8_bit_rows_of_any_length(rows, D, dtype):
    """More rows than a grid has teams or warps, at every place of a 16-byte chunk: the norm's output within its bound, the
    quantised rows to the bit, and both products' inputs alike."""
    gen = torch.Generator().manual_seed(rows)
    x, res = (torch.randn(rows, D, generator=gen).to(dtype).cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(D, generator=gen)).cuda()
    q, c, s = gdn.rms_norm_fp8(x, w, residual=res)
    assert torch.equal(s, (x.float() + res.float()).to(dtype))
    (y, _), (e, _) = ref.rms_fwd(s, w, 1e-5)
    ref.check_e4m3(q, ref.spread(c, rows, D, 1), y, 2 * e, "norm")
    q, c = gdn.fp8_quantize(x)
    want_c = ref.scales(x, 1).float().clamp(min=ref.TINY) / 448
    u = x.cpu().float() / ref.spread(want_c, rows, D, 1).float()
    assert torch.equal(c.cpu(), want_c) and same(q.cpu(), u.clamp(-448, 448).to(torch.float8_e4m3fn))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_log_probability_gradients_below_the_normal_numbers(dtype):
    """Rows whose gradients lie below 2^-126, where their reciprocals and their small multiples are no fp32 numbers, beside
    ordinary ones: nothing infinite or NaN comes of them, the other rows' results stay as they are, and their own dh is the
    formula's.  On the CUDA cores the logits' gradient itself is a multiple of 2^-149 then, three operations of up to half a
    step each; on the tensor cores it is in units of the row's weight."""
    gen = torch.Generator().manual_seed(8)
    T = torch.float32 if dtype == "f32" else torch.bfloat16
    N, D, V = 40, 32, 300
    h, w = (0.5 * torch.randn(n, D, generator=gen) for n in (N, V))
    h, w, t = h.to(T).cuda(), w.to(T).cuda(), torch.randint(0, V, (N,), generator=gen).to(torch.int32).cuda()
    _, H, lse, _, _ = gdn.linear_log_probs_fwd(h, w, t)
    small = torch.tensor([1e-39, -2e-40, 2.0 ** -149, 0.0, 0.0, 1e-39])
    other = torch.tensor([0.0, 1e-39, 2.0 ** -149, 1e-40, 2.0 ** -140, 1e-45])
    da, db = torch.ones(N), 0.1 * torch.ones(N)
    da[:6], db[:6] = small, other
    da, db = da.cuda(), db.cuda()
    dh, dw = gdn.linear_log_probs_bwd(h, w, t, lse, H, da, db)
    assert torch.isfinite(dh.float()).all() and torch.isfinite(dw.float()).all() and (dh[:6].float().abs() < 1e-37).all()
    da0, db0 = da.clone(), db.clone()
    da0[:6], db0[:6] = 0, 0
    dh0, dw0 = gdn.linear_log_probs_bwd(h, w, t, lse, H, da0, db0)
    assert torch.equal(dw, dw0) and torch.equal(dh[6:], dh0[6:]) and (dh0[:6] == 0).all()
    # a weight larger by what h is smaller leaves the logits and takes dh into the normal numbers
    up, down = (w.float() * 2.0 ** 60).to(T), (h.float() * 2.0 ** -60).to(T)
    dh, _ = gdn.linear_log_probs_bwd(down, up, t, lse, H, da, db)
    want, bound = ref.log_probs_bwd(down, up, t, lse, H, da, db, low_bits=dtype == "bf16")
    room = bound[0] + (ref.BF16 * want[0].abs() * 1.01 if dtype == "bf16" else 2.0 ** -148 * ref.f64(up).abs().sum(0) + ref.U * want[0].abs())
    err = (ref.f64(dh) - want[0]).abs()
    assert (err[:6] <= room[:6]).all(), (err / room.clamp(min=1e-300))[:6].max(-1).values
