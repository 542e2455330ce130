"""More operators around the gated delta rule layer, as measured cases: root-mean-square norm with the residual's addition
(forward, backward, and with an output in 8 bits), the matrix product of 8-bit operands with a scale for each block of 128, with
its quantising, and the log probabilities of given tokens with entropy and top alternatives, forward and backward.

    s = x + r,  y = s rstd w,  rstd = (mean s^2 + eps)^(-1/2)                                 (norm; s is rounded as it is stored)
    q = e4m3(y / c),  c = max |y| / 448 over each 128 columns                                 (8 bits; weights: each 128 x 128)
    out_mn = sum_b c_mb d_{n/128,b} sum_{k in b} q_mk w_nk                                     (product of 8-bit operands)
    logp_i = l_{i,t_i} - lse_i,  H_i = lse_i - sum_v p_iv l_iv,  l = h w'                      (log probabilities, entropy)
    dl_iv = a_i ([v = t_i] - p_iv) - b_i p_iv (log p_iv + H_i)  for gradients a, b of them
A row whose target is outside [0, V) is ignored: its results are 0, its alternatives' ids -1.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK, E4M3_MAX, TINY = 128, 448.0, 2.0 ** -100


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(op, rows, D, dtype, residual=True, **kw):
    return dict(op=op, rows=rows, D=D, dtype=dtype, residual=residual, **kw)


def _quant(rows, D, dtype, block_rows, **kw):
    return dict(op="quantize", rows=rows, D=D, dtype=dtype, block_rows=block_rows, **kw)


def _linear(tokens, K, N, **kw):
    return dict(op="fp8_linear", tokens=tokens, K=K, N=N, dtype="bf16", **kw)


def _logp(op, tokens, D, vocab, top=0, entropy=True, **kw):
    return dict(op=op, tokens=tokens, D=D, vocab=vocab, top=top, entropy=entropy, dtype="bf16", **kw)


def listed():
    return [
        # a few short rows of an odd width, as in a small model or a test: launch latency
        _norm("rms_fwd", 300, 1001, "f32", name="rms_fwd_300x1001_f32"),
        # the norm before each mixer with the sum of the residual stream, headline batch
        _norm("rms_fwd", 8192, 2048, "bf16", name="rms_fwd_8192x2048_bf16"),
        # its training backward, the later layers' gradient of the stream added
        _norm("rms_bwd", 8192, 2048, "bf16", name="rms_bwd_8192x2048_bf16"),
        # in front of the 8-bit projections: one decode token for 256 sequences, and the prefill of the headline batch
        _norm("rms_fp8", 256, 2048, "bf16", name="rms_fp8_256x2048_bf16"),
        _norm("rms_fp8", 8192, 2048, "bf16", name="rms_fp8_8192x2048_bf16"),
        # the mixer's output, 16 heads of 128, on its way into the 8-bit output projection
        _quant(8192, 2048, "bf16", 1, name="quantize_8192x2048_bf16"),
        # the projection of q, k and v (16 heads of 128 each): one token, a decode batch, the prefill of the headline batch
        _linear(1, 2048, 6144, name="fp8_linear_1x2048x6144"),
        _linear(256, 2048, 6144, name="fp8_linear_256x2048x6144"),
        _linear(8192, 2048, 6144, name="fp8_linear_8192x2048x6144"),
        # scoring a few hundred tokens against a vocabulary of an odd size, with the alternatives a client asks for
        _logp("logp_fwd", 255, 1024, 50257, top=8, name="logp_fwd_255x1024x50257_top8"),
        # scoring the headline batch
        _logp("logp_fwd", 8192, 2048, 32768, top=5, name="logp_fwd_8192x2048x32768_top5"),
        # the gradient of a policy's loss with an entropy bonus over the same batch: the largest case
        _logp("logp_bwd", 8192, 2048, 32768, name="logp_bwd_8192x2048x32768"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rms_fwd", "rms_bwd", "rms_fp8", "quantize", "fp8_linear", "fp8_linear", "logp_fwd", "logp_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("rms_fwd", "rms_bwd", "rms_fp8", "quantize"):
        D = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            D = -(-D // 8) * 8
        rows = min(_log(rng, 1, 131072), (32 << 20) // D)
        if kind == "quantize":
            return _quant(rows, D, dtype, rng.choice([1, 128]))
        return _norm(kind, rows, D, dtype, residual=rng.random() < 0.75)
    if kind == "fp8_linear":
        K, N = 16 * _log(rng, 4, 512), _log(rng, 16, 16384)
        if rng.random() < 0.5:
            N = -(-N // 64) * 64
        tokens = _log(rng, 1, 8192)
        return _linear(max(1, min(tokens, (8192 * 2048 * 6144) // (K * N))), K, N)
    D, vocab = 8 * _log(rng, 8, 256), _log(rng, 17, 65536)
    tokens = max(1, min(_log(rng, 1, 8192), (8192 * 2048 * 32768) // (D * vocab)))
    if kind == "logp_fwd":
        return _logp(kind, tokens, D, vocab, top=rng.choice([0, 1, 5, 8, 17]))
    return _logp(kind, tokens, D, vocab, entropy=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _dt(case), case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rows(n, D):
        # rows of a residual stream: unequal scales, a few loud channels
        x = randn(n, D) * torch.exp(0.5 * randn(n, 1))
        x[:, :: max(1, D // 4)] *= 4
        return x

    s = dict(case)
    if op in ("rms_fwd", "rms_fp8"):
        s["x"] = randn(case["rows"], case["D"]).to(dt)                       # what the last layer adds
        s["r"] = rows(case["rows"], case["D"]).to(dt) if case["residual"] else None
        s["w"] = 1 + 0.1 * randn(case["D"])
    elif op == "rms_bwd":
        s["x"] = rows(case["rows"], case["D"]).to(dt)                        # the sum that the forward pass stored
        s["w"] = 1 + 0.1 * randn(case["D"])
        s["rstd"] = _rms(s["x"])
        s["dout"] = randn(case["rows"], case["D"]).to(dt)
        s["dres"] = randn(case["rows"], case["D"]).to(dt) if case["residual"] else None
    elif op == "quantize":
        s["x"] = rows(case["rows"], case["D"]).to(dt)
    elif op == "fp8_linear":
        M, K, N = case["tokens"], case["K"], case["N"]
        s["x"], s["xc"] = _quantize(rows(M, K), 1)
        s["w"], s["wc"] = _quantize(randn(N, K) * K ** -0.5, BLOCK)
    else:
        # Values on a grid, as many bits as bf16 weights hold, so that the logits' sums are exact in 32 bits whatever their
        # order: the alternatives' ids then go by the inputs alone, equal logits (there are some) by the lower index.
        N, D, V = case["tokens"], case["D"], case["vocab"]
        scale = 2.0 ** -round(math.log2(math.sqrt(D) / 2))
        s["h"] = ((16 * randn(N, D)).round().clamp(-64, 64) / 16).to(dt)
        s["w"] = ((16 * randn(V, D)).round().clamp(-64, 64) / 16 * scale).to(dt)
        t = torch.randint(0, V, (N,), generator=gen, device="cuda")
        t[torch.rand(N, generator=gen, device="cuda") < 0.03] = -100         # padding and prompt tokens
        s["t"] = t.to(torch.int32)
        if op == "logp_bwd":
            f = _logp_fwd({**s, "top": 0})
            s["H"], s["lse"] = f[1], f[2]
            kept = (t >= 0).sum().clamp(min=1)
            s["dlogp"] = randn(N) / kept                                     # advantages, of both signs
            s["dent"] = torch.full((N,), 0.01, device="cuda") / kept if case["entropy"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rms(s):
    return torch.rsqrt(s.float().square().mean(-1) + EPS)


def _sum(s):
    return s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)


def _rms_fwd(s):
    t = _sum(s)
    rstd = _rms(t)
    y = (t.float() * rstd[:, None] * s["w"]).to(t.dtype)
    return (y, rstd) if s["r"] is None else (y, t, rstd)


def _rms_bwd(s):
    xhat = s["x"].float() * s["rstd"][:, None]
    dy = s["dout"].float()
    u = dy * s["w"]
    dx = s["rstd"][:, None] * (u - xhat * (u * xhat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(0)


def _quantize(y, block_rows):
    """[R, D] fp32 to e4m3 and the scales of its blocks of block_rows x 128."""
    R, D = y.shape
    R1, D1 = -(-R // block_rows), -(-D // BLOCK)
    p = torch.zeros((R1 * block_rows, D1 * BLOCK), device=y.device)
    p[:R, :D] = y
    p = p.view(R1, block_rows, D1, BLOCK)
    c = p.abs().amax((1, 3)).clamp(min=TINY) / E4M3_MAX
    q = (p / c[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(R1 * block_rows, D1 * BLOCK)[:R, :D].contiguous(), c


def _rms_fp8(s):
    t = _sum(s)
    q, c = _quantize(t.float() * _rms(t)[:, None] * s["w"], 1)
    return (q, c) if s["r"] is None else (q, c, t)


def _blocks(c, R, D, block_rows):
    """The scales [R1, D1] laid out for each value of [R, D]."""
    return c.repeat_interleave(block_rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :D]


def _fp8_linear(s):
    M, K, N = s["tokens"], s["K"], s["N"]
    x = s["x"].float() * _blocks(s["xc"], M, K, 1)
    w = s["w"].float() * _blocks(s["wc"], N, K, BLOCK)
    return (x @ w.T).to(torch.bfloat16)


def _logp_fwd(s):
    V, k = s["vocab"], min(s["top"], s["vocab"])
    logits = s["h"].float() @ s["w"].float().T
    kept = (s["t"] >= 0) & (s["t"] < V)
    top = logits.max(-1).values
    z = logits - top[:, None]
    p = torch.exp(z)
    sum_p = p.sum(-1)
    lse = top + torch.log(sum_p)
    at = logits.gather(1, torch.where(kept, s["t"], 0).long()[:, None])[:, 0]
    logp, H = at - lse, torch.log(sum_p) - (p * z).sum(-1) / sum_p
    out = [torch.where(kept, v, 0.0) for v in (logp, H, lse)]
    if k:
        # one whole number a word, ordered by its logit and then by the lower index
        bits = (logits + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) * (1 << 24) - torch.arange(V, device=logits.device)
        ids = torch.topk(key, k, -1).indices
        out += [torch.where(kept[:, None], ids, -1).int(),
                torch.where(kept[:, None], logits.gather(1, ids) - lse[:, None], 0.0)]
    return out


def _logp_bwd(s):
    h, w = s["h"].float(), s["w"].float()
    kept = ((s["t"] >= 0) & (s["t"] < s["vocab"]))[:, None]
    lp = h @ w.T - s["lse"][:, None]
    p = torch.exp(lp)
    g = -s["dlogp"][:, None] * p
    if s["dent"] is not None:
        g = g - s["dent"][:, None] * p * (lp + s["H"][:, None])
    g.scatter_add_(1, torch.where(kept, s["t"][:, None], 0).long(), s["dlogp"][:, None].contiguous())
    g = torch.where(kept, g, 0.0)
    return (g @ w).to(s["h"].dtype), (g.T @ h).to(s["w"].dtype)


def run(s):
    op = s["op"]
    if not own:
        if op == "quantize":
            return _quantize(s["x"].float(), s["block_rows"])
        return {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "rms_fp8": _rms_fp8, "fp8_linear": _fp8_linear,
                "logp_fwd": _logp_fwd, "logp_bwd": _logp_bwd}[op](s)
    import gated_delta_rule_12_gb300 as gdn
    if op == "rms_fwd":
        y, t, rstd = gdn.rms_norm_fwd(s["x"], s["w"], residual=s["r"], eps=EPS)
        return (y, rstd) if t is None else (y, t, rstd)
    if op == "rms_bwd":
        return gdn.rms_norm_bwd(s["dout"], s["x"], s["rstd"], s["w"], dresidual=s["dres"])
    if op == "rms_fp8":
        q, c, t = gdn.rms_norm_fp8(s["x"], s["w"], residual=s["r"], eps=EPS)
        return (q, c) if t is None else (q, c, t)
    if op == "quantize":
        return gdn.fp8_quantize(s["x"], block_rows=s["block_rows"])
    if op == "fp8_linear":
        return gdn.fp8_linear(s["x"], s["xc"], s["w"], s["wc"])
    if op == "logp_fwd":
        k = min(s["top"], s["vocab"])
        logp, H, lse, ids, top = gdn.linear_log_probs_fwd(s["h"], s["w"], s["t"], top_k=k)
        return [logp, H, lse, ids, top] if k else [logp, H, lse]
    return gdn.linear_log_probs_bwd(s["h"], s["w"], s["t"], s["lse"], s["H"], s["dlogp"], s["dent"])


def work(case):
    op, z = case["op"], _size(case)
    if op in ("rms_fwd", "rms_bwd", "rms_fp8", "quantize"):
        R, D = case["rows"], case["D"]
        E, scales = R * D, 4 * R * -(-D // BLOCK)
        if op == "quantize":
            return {"bytes": E * (z + 1) + scales // case["block_rows"], "flops": 3 * E}
        res = case["residual"]
        if op == "rms_fwd":
            return {"bytes": (4 if res else 2) * E * z + 4 * R + 4 * D, "flops": 5 * E}
        if op == "rms_fp8":
            return {"bytes": E * ((3 if res else 1) * z + 1) + scales + 4 * D, "flops": 8 * E}
        return {"bytes": (4 if res else 3) * E * z + 4 * R + 8 * D, "flops": 10 * E}
    if op == "fp8_linear":
        M, K, N = case["tokens"], case["K"], case["N"]
        KB, NB = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": (M + N) * K + 4 * (M + NB) * KB + 2 * M * N, "flops": 2 * M * N * K}
    N, D, V = case["tokens"], case["D"], case["vocab"]
    read = (N + V) * D * z
    if op == "logp_fwd":
        return {"bytes": read + 16 * N + 8 * N * min(case["top"], V), "flops": 2 * N * V * D}
    return {"bytes": 2 * read + 20 * N, "flops": 6 * N * V * D}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def _quantize64(y, block_rows):
    """Value by value: each one's scale is its block's, found by index."""
    R, D = y.shape
    dev = y.device
    i, j = torch.arange(R, device=dev) // block_rows, torch.arange(D, device=dev) // BLOCK
    c = torch.full((int(i[-1]) + 1, int(j[-1]) + 1), TINY, dtype=torch.float64, device=dev)
    at = i[:, None] * c.shape[1] + j
    c.view(-1).scatter_reduce_(0, at.view(-1), y.abs().reshape(-1), "amax")
    c /= E4M3_MAX
    u = y / c.view(-1)[at]
    # e4m3: steps of 2^-3 of the value's power of two, 2^-9 at least
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step, c


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and "float" in str(v.dtype)}
    if op == "quantize":
        return _quantize64(f["x"], case["block_rows"])
    if op in ("rms_fwd", "rms_fp8"):
        t = f["x"] if s["r"] is None else (f["x"] + f["r"]).to(s["x"].dtype).double()
        n = (torch.einsum("rd,rd->r", t, t) / case["D"] + EPS).sqrt()
        y = t / n[:, None] * f["w"]
        more = () if s["r"] is None else (t,)
        if op == "rms_fwd":
            return (y, *more, 1 / n)
        return (*_quantize64(y, 1), *more)
    if op == "rms_bwd":
        # the gradient as a projection: dx is rstd (I - xhat xhat'/D) (dy w), with the given statistics
        xhat = f["rstd"][:, None] * f["x"]
        u = f["dout"] * f["w"]
        dx = f["rstd"][:, None] * u - (f["rstd"] * torch.einsum("rd,rd->r", u, xhat) / case["D"])[:, None] * xhat
        return dx + f.get("dres", 0.0), torch.einsum("rd,rd->d", f["dout"], xhat)
    if op == "fp8_linear":
        M, K, N = case["tokens"], case["K"], case["N"]
        out = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        rows = torch.arange(N, device="cuda") // BLOCK
        for b in range(-(-K // BLOCK)):
            k = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
            out += (f["x"][:, k] @ f["w"][:, k].T) * f["xc"][:, b, None] * f["wc"][rows, b]
        return out
    N, V, top = case["tokens"], case["vocab"], min(case["top"], case["vocab"])
    h, w, t = f["h"], f["w"], s["t"].long()
    kept = (t >= 0) & (t < V)
    if op == "logp_fwd":
        logp, H, lse = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(3))
        ids = torch.full((N, top), -1, dtype=torch.int32, device="cuda")
        best = torch.zeros((N, top), dtype=torch.float64, device="cuda")
        for i in range(0, N, 512):
            k = kept[i:i + 512].nonzero()[:, 0] + i
            if not len(k):
                continue
            lp = torch.log_softmax(h[k] @ w.T, -1)
            logp[k] = lp[torch.arange(len(k), device="cuda"), t[k]]
            H[k] = -(lp.exp() * lp).sum(-1)
            lse[k] = torch.logsumexp(h[k] @ w.T, -1)
            if top:
                v, at = torch.sort(lp, dim=-1, descending=True, stable=True)
                best[k], ids[k] = v[:, :top], at[:, :top].int()
        return [logp, H, lse, ids, best] if top else [logp, H, lse]
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for i in range(0, N, 512):
        k = kept[i:i + 512].nonzero()[:, 0] + i
        if not len(k):
            continue
        lp = h[k] @ w.T - f["lse"][k][:, None]
        p = lp.exp()
        g = -p
        g[torch.arange(len(k), device="cuda"), t[k]] += 1
        g *= f["dlogp"][k][:, None]
        if s["dent"] is not None:
            g -= f["dent"][k][:, None] * p * (lp + f["H"][k][:, None])
        dh[k] = g @ w
        dw += g.T @ h[k]
    return dh, dw
