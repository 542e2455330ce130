"""The operators around the gated delta rule layer, as measured cases: the per-channel gated scan, layer norm and the
linear softmax cross entropy, each forward and backward, the scan for single tokens too.

    h_t = a_t h_{t-1} + c_t x_t,  a = exp(g),  c = 1, or 1 - a with the input gate            (gated scan)
    y   = (x - mean) rstd w + b,  over the last axis                                         (layer norm)
    loss_i = log sum_v exp(h_i . w_v) - h_i . w_{t_i}; targets outside [0, V) are ignored     (linear cross entropy)
"""
import math

import torch

own = False

EPS = 1e-5


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _scan(op, seqs, tokens, D, dtype, packed=False, init=False, input_gate=False, **kw):
    """`seqs` sequences of `tokens` tokens each, or `tokens` tokens in all where they are packed."""
    return dict(op=op, seqs=seqs, tokens=tokens, D=D, dtype=dtype, packed=packed, init=init, input_gate=input_gate, **kw)


def _norm(op, rows, D, dtype, **kw):
    return dict(op=op, rows=rows, D=D, dtype=dtype, **kw)


def _ce(op, tokens, D, vocab, **kw):
    return dict(op=op, tokens=tokens, D=D, vocab=vocab, dtype="bf16", **kw)


def listed():
    return [
        # one decode token for 256 sequences, 16 x 128 channels: the library's decode batch
        _scan("scan_step", 256, 1, 2048, "bf16", init=True, name="scan_step_n256_d2048_bf16"),
        # prefill or training forward at the library's headline batch
        _scan("scan_fwd", 4, 2048, 2048, "bf16", name="scan_fwd_b4_l2048_d2048_bf16"),
        # packed prefill with carried states: the library's varlen workload
        _scan("scan_fwd", 8, 32768, 2048, "bf16", packed=True, init=True, name="scan_fwd_packed_32768_d2048_bf16"),
        # the training backward of the headline batch
        _scan("scan_bwd", 4, 2048, 2048, "bf16", name="scan_bwd_b4_l2048_d2048_bf16"),
        # one long sequence of odd sizes in fp32 with an input gate: little parallelism but along time
        _scan("scan_bwd", 1, 4999, 1001, "f32", init=True, input_gate=True, name="scan_bwd_b1_l4999_d1001_f32"),
        # a few short rows of an odd width, as in a small model or a test: launch latency
        _norm("norm_fwd", 300, 1001, "f32", name="norm_fwd_300x1001_f32"),
        # the norm before each mixer, headline batch
        _norm("norm_fwd", 8192, 2048, "bf16", name="norm_fwd_8192x2048_bf16"),
        _norm("norm_bwd", 8192, 2048, "bf16", name="norm_bwd_8192x2048_bf16"),
        # the per-head norm behind the mixer: 16 heads of 128 for each of 8192 tokens
        _norm("norm_bwd", 131072, 128, "bf16", name="norm_bwd_131072x128_bf16"),
        # scoring a few hundred tokens against a vocabulary of an odd size: one read of the weights
        _ce("ce_fwd", 255, 1024, 50257, name="ce_fwd_255x1024x50257_bf16"),
        # evaluation and training loss of the headline batch
        _ce("ce_fwd", 8192, 2048, 32768, name="ce_fwd_8192x2048x32768_bf16"),
        # its gradient over a large vocabulary: the largest case
        _ce("ce_bwd", 8192, 2048, 65536, name="ce_bwd_8192x2048x65536_bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd", "ce_fwd", "ce_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "scan_step":
        return _scan(kind, _log(rng, 1, 1024), 1, _log(rng, 16, 8192), dtype, init=True, input_gate=rng.random() < 0.3)
    if kind in ("scan_fwd", "scan_bwd"):
        D = _log(rng, 16, 4096)
        if rng.random() < 0.5:
            D = -(-D // 8) * 8
        packed = rng.random() < 0.4
        tokens = _log(rng, 1, 32768)
        seqs = _log(rng, 1, 16)
        limit = 64 << 20   # elements: the packed workload's
        tokens = min(tokens, max(1, limit // (D * (1 if packed else seqs))))
        return _scan(kind, seqs, tokens, D, dtype, packed=packed, init=rng.random() < 0.5, input_gate=rng.random() < 0.3)
    if kind in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            D = -(-D // 8) * 8
        return _norm(kind, min(_log(rng, 1, 131072), (32 << 20) // D), D, dtype)
    D = 8 * _log(rng, 8, 256)
    return _ce(kind, _log(rng, 1, 8192), D, _log(rng, 17, 65536))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _dt(case), case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = dict(case)
    if op.startswith("scan"):
        D, N, T = case["D"], case["seqs"], case["tokens"]
        lead = (1, T) if case["packed"] else (N, T)
        if op == "scan_step":
            lead = (N,)
        if case["packed"]:   # sequences of unequal lengths, some of them perhaps empty
            host = torch.Generator().manual_seed(seed)
            cut = torch.randint(0, T + 1, (N - 1,), generator=host).sort().values
            s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([T])]).to("cuda", torch.int32)
        else:
            s["cu"] = None
        s["x"] = randn(*lead, D).to(dt)
        # log-decays as the library's workloads draw them: -0.1 softplus(z)
        s["g"] = (-0.1 * torch.log1p(torch.exp(randn(*lead, D)))).to(dt)
        s["state"] = 0.5 * randn(N, D) if case["init"] else None
        if op == "scan_bwd":
            # what the forward call returned: h, rounded to the element type
            s["out"] = _scan_fwd(s)[0]
            s["dout"] = randn(*lead, D).to(dt)
            s["dfinal"] = randn(N, D) if case["init"] else None
    elif op.startswith("norm"):
        rows, D = case["rows"], case["D"]
        # rows of a residual stream: unequal scales, a common offset, a few loud channels
        x = randn(rows, D) * torch.exp(0.5 * randn(rows, 1)) + 0.3 * randn(rows, 1)
        x[:, :: max(1, D // 4)] *= 4
        s["x"] = x.to(dt)
        s["w"], s["b"] = 1 + 0.1 * randn(D), 0.1 * randn(D)
        if op == "norm_bwd":
            _, s["mean"], s["rstd"] = _norm_fwd(s)
            s["dout"] = randn(rows, D).to(dt)
    else:
        N, D, V = case["tokens"], case["D"], case["vocab"]
        s["h"] = randn(N, D).to(dt)
        s["w"] = (randn(V, D) * (2 * D ** -0.5)).to(dt)
        t = torch.randint(0, V, (N,), generator=gen, device="cuda")
        t[torch.rand(N, generator=gen, device="cuda") < 0.03] = -100   # padding and prompt tokens
        s["t"] = t.to(torch.int32)
        if op == "ce_bwd":
            _, s["lse"] = _ce_fwd(s)
            kept = (t >= 0).sum().clamp(min=1)
            s["dloss"] = torch.ones(N, device="cuda") / kept          # the gradient of a mean over the kept tokens
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _tokens(s):
    """For each token of the flattened axis: its sequence, and whether it is that sequence's first or last; and the
    sequences' bounds."""
    dev = s["x"].device
    if s["cu"] is None:
        cu = torch.arange(s["seqs"] + 1, device=dev) * s["tokens"]
    else:
        cu = s["cu"].long()
    t = torch.arange(s["x"].numel() // s["D"], device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, (t == cu[seq])[:, None], (t + 1 == cu[seq + 1])[:, None], cu


def _scan_doubling(a, u):
    """h_t = a_t h_{t-1} + u_t along the first axis from h = 0, in log2(T) steps of pairwise composition."""
    step = 1
    while step < u.shape[0]:
        u = torch.cat([u[:step], u[step:] + a[step:] * u[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return u


def _coef(g, input_gate):
    a = torch.exp(g)
    return a, (-torch.expm1(g) if input_gate else torch.ones_like(a))


def _scan_fwd(s):
    D, dt = s["D"], s["x"].dtype
    x, g = s["x"].float().reshape(-1, D), s["g"].float().reshape(-1, D)
    seq, first, _, cu = _tokens(s)
    a, c = _coef(g, s["input_gate"])
    u = c * x
    state = s["state"] if s["state"] is not None else torch.zeros((s["seqs"], D), device=x.device)
    u = torch.where(first, u + a * state[seq], u)
    h = _scan_doubling(torch.where(first, 0.0, a), u)
    final = torch.where((cu[1:] > cu[:-1])[:, None], h[(cu[1:] - 1).clamp(min=0)], state)
    return h.to(dt).reshape(s["x"].shape), final


def _scan_bwd(s):
    D, dt = s["D"], s["x"].dtype
    x, g, h, do = (s[n].float().reshape(-1, D) for n in ("x", "g", "out", "dout"))
    seq, first, last, cu = _tokens(s)
    a, c = _coef(g, s["input_gate"])
    zero = torch.zeros((s["seqs"], D), device=x.device)
    state = s["state"] if s["state"] is not None else zero
    df = s["dfinal"] if s["dfinal"] is not None else zero
    do = torch.where(last, do + df[seq], do)
    # e_t = a_t (do_t + e_{t+1}) is the gradient of h_{t-1}: the same scan, from the end
    e = _scan_doubling(torch.where(last, 0.0, a).flip(0), (a * do).flip(0)).flip(0)
    dh = torch.where(last, do, do + torch.cat([e[1:], e[:1]]))
    before = torch.where(first, state[seq], torch.cat([h[:1], h[:-1]]))
    dx = c * dh
    dg = a * dh * (before - x if s["input_gate"] else before)
    out = [dx.to(dt).reshape(s["x"].shape), dg.to(dt).reshape(s["x"].shape)]
    if s["state"] is not None:
        out.append(torch.where((cu[1:] > cu[:-1])[:, None], e[cu[:-1].clamp(max=e.shape[0] - 1)], df))
    return out


def _scan_step(s):
    a, c = _coef(s["g"].float(), s["input_gate"])
    s["state"].copy_(a * s["state"] + c * s["x"].float())
    return s["state"].to(s["x"].dtype), s["state"]


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(-1) + EPS)
    return (d * rstd[:, None] * s["w"] + s["b"]).to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dout"].float()
    u = dy * s["w"]
    dx = s["rstd"][:, None] * (u - u.mean(-1, keepdim=True) - xhat * (u * xhat).mean(-1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _ce_fwd(s):
    logits = s["h"].float() @ s["w"].float().T
    kept = (s["t"] >= 0) & (s["t"] < s["vocab"])
    top = logits.max(-1).values
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(-1))
    at = logits.gather(1, torch.where(kept, s["t"], 0).long()[:, None])[:, 0]
    return torch.where(kept, lse - at, 0.0), torch.where(kept, lse, 0.0)


def _ce_bwd(s):
    h, w = s["h"].float(), s["w"].float()
    kept = (s["t"] >= 0) & (s["t"] < s["vocab"])
    p = torch.exp(h @ w.T - s["lse"][:, None])
    at = torch.where(kept, s["t"], 0).long()[:, None]
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=p.dtype))
    p = torch.where(kept[:, None], p * s["dloss"][:, None], 0.0)
    return (p @ w).to(s["h"].dtype), (p.T @ h).to(s["w"].dtype)


def run(s):
    op = s["op"]
    if not own:
        return {"scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd, "scan_step": _scan_step, "norm_fwd": _norm_fwd,
                "norm_bwd": _norm_bwd, "ce_fwd": _ce_fwd, "ce_bwd": _ce_bwd}[op](s)
    import gated_delta_rule_12_gb300 as gdn
    if op == "scan_fwd":
        return gdn.gated_scan_fwd(s["x"], s["g"], init_state=s["state"], cu_seqlens=s["cu"], input_gate=s["input_gate"])
    if op == "scan_bwd":
        dx, dg, dinit = gdn.gated_scan_bwd(s["x"], s["g"], s["out"], s["dout"], init_state=s["state"],
                                           dfinal_state=s["dfinal"], cu_seqlens=s["cu"], input_gate=s["input_gate"],
                                           want_dinit=s["state"] is not None)
        return [dx, dg] if dinit is None else [dx, dg, dinit]
    if op == "scan_step":
        return gdn.gated_scan_step(s["state"], s["x"], s["g"], input_gate=s["input_gate"]), s["state"]
    if op == "norm_fwd":
        return gdn.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_bwd":
        return gdn.layer_norm_bwd(s["dout"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "ce_fwd":
        return gdn.linear_cross_entropy_fwd(s["h"], s["w"], s["t"])
    return gdn.linear_cross_entropy_bwd(s["h"], s["w"], s["t"], s["lse"], s["dloss"])


def work(case):
    op, z = case["op"], _size(case)
    if op.startswith("scan"):
        N, D = case["seqs"], case["D"]
        E = D * case["tokens"] * (1 if case["packed"] else N)
        states = 4 * N * D
        if op == "scan_step":
            return {"bytes": 3 * E * z + 2 * states, "flops": 3 * E}
        if op == "scan_fwd":
            return {"bytes": 3 * E * z + states * (2 if case["init"] else 1), "flops": 3 * E}
        return {"bytes": (6 if case["input_gate"] else 5) * E * z + (3 * states if case["init"] else 0), "flops": 6 * E}
    if op.startswith("norm"):
        rows, D = case["rows"], case["D"]
        if op == "norm_fwd":
            return {"bytes": 2 * rows * D * z + 8 * rows + 8 * D, "flops": 7 * rows * D}
        return {"bytes": 3 * rows * D * z + 8 * rows + 12 * D, "flops": 12 * rows * D}
    N, D, V = case["tokens"], case["D"], case["vocab"]
    read = (N + V) * D * z + 12 * N
    if op == "ce_fwd":
        return {"bytes": read, "flops": 2 * N * V * D}
    return {"bytes": 2 * read, "flops": 6 * N * V * D}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "scan_step":
        a = f["g"].exp()
        h = a * f["state"] + ((1 - a) if case["input_gate"] else 1.0) * f["x"]
        return h, h
    if op.startswith("scan"):
        N, D, T = case["seqs"], case["D"], case["tokens"]
        bounds = s["cu"].tolist() if s["cu"] is not None else [n * T for n in range(N + 1)]
        flat = {k: f[k].reshape(-1, D) for k in ("x", "g", "out", "dout") if k in f}
        a = flat["g"].exp()
        c = 1 - a if case["input_gate"] else torch.ones_like(a)
        zero = torch.zeros(N, D, dtype=torch.float64, device="cuda")
        state = f.get("state", zero)
        # one step at a time; sequences of equal lengths advance together
        if case["packed"]:
            rows = [(bounds[n], bounds[n + 1] - bounds[n], slice(n, n + 1), 1) for n in range(N)]
        else:
            rows = [(0, T, slice(0, N), N)]
        if op == "scan_fwd":
            out, final = torch.empty_like(a), state.clone()
            for at, length, ns, m in rows:
                view = lambda v: v[at:at + length * m].view(m, length, D)  # noqa: E731
                h, u, aa, o = state[ns].clone(), view(c * flat["x"]), view(a), view(out)
                for t in range(length):
                    h = torch.addcmul(u[:, t], aa[:, t], h)
                    o[:, t] = h
                final[ns] = h
            return out.view(s["x"].shape), final
        df = f.get("dfinal", zero)
        dx, dg, dinit = torch.empty_like(a), torch.empty_like(a), df.clone()
        for at, length, ns, m in rows:
            view = lambda v: v[at:at + length * m].view(m, length, D)  # noqa: E731
            e, aa, do, dd = df[ns].clone(), view(a), view(flat["dout"]), torch.empty(m, length, D, dtype=torch.float64, device="cuda")
            for t in range(length - 1, -1, -1):
                dd[:, t] = do[:, t] + e
                e = aa[:, t] * dd[:, t]
            prev = torch.cat([state[ns][:, None], view(flat["out"])[:, :-1]], 1)[:, :length]
            view(dx).copy_(view(c) * dd)
            view(dg).copy_(aa * dd * (prev - (view(flat["x"]) if case["input_gate"] else 0.0)))
            dinit[ns] = e
        return [dx.view(s["x"].shape), dg.view(s["x"].shape)] + ([dinit] if case["init"] else [])
    if op.startswith("norm"):
        x, w, b = f["x"], f["w"], f["b"]
        if op == "norm_fwd":
            var, mean = torch.var_mean(x, -1, unbiased=False)
            rstd = (var + EPS) ** -0.5
            return (x - mean[:, None]) / (var + EPS).sqrt()[:, None] * w + b, mean, rstd
        # the gradient as a projection: dx is rstd (I - 11'/D - xhat xhat'/D) (dy w), with the given statistics
        D, r, dy = case["D"], f["rstd"][:, None], f["dout"]
        xhat = r * (x - f["mean"][:, None])
        u = dy * w
        dx = r * u - r / D * (u.sum(-1, keepdim=True) + xhat * torch.einsum("rd,rd->r", u, xhat)[:, None])
        return dx, torch.einsum("rd,rd->d", dy, xhat), dy.sum(0)
    N, V = case["tokens"], case["vocab"]
    if N * V * case["D"] > 3 << 40:
        return None
    h, w, t = f["h"], f["w"], s["t"].long()
    kept = (t >= 0) & (t < V)
    if op == "ce_fwd":
        loss, lse = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
        for i in range(0, N, 1024):
            logits = h[i:i + 1024] @ w.T
            k = kept[i:i + 1024]
            lse[i:i + 1024] = torch.where(k, torch.logsumexp(logits, -1), 0.0)
            picked = logits[torch.arange(len(k), device="cuda"), t[i:i + 1024].clamp(0, V - 1)]
            loss[i:i + 1024] = torch.where(k, lse[i:i + 1024] - picked, 0.0)
        return loss, lse
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for i in range(0, N, 1024):
        k = kept[i:i + 1024].nonzero()[:, 0] + i
        if not len(k):
            continue
        p = torch.exp(h[k] @ w.T - f["lse"][k][:, None])
        p[torch.arange(len(k), device="cuda"), t[k]] -= 1
        p *= f["dloss"][k][:, None]
        dh[k] = p @ w
        dw += p.T @ h[k]
    return dh, dw
