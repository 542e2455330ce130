"""64-bit plain forms of the root-mean-square norm, the 8-bit quantising and product, on the CPU, and the error bounds
that the kernels are held to, counted as in ops_reference: roundings times a magnitude evaluated in 64 bits.  Nothing
here is shared with the library."""
import torch

from ops_reference import BF16, U, check, f64  # noqa: F401

E4M3_MAX, TINY = 448.0, 2.0 ** -100


def rms_fwd(s, w, eps):
    """(out, rstd) of the rows s as they are stored, and bounds.  The squares' sum has positive terms and at most
    D / 32 + 16 roundings on a path; rstd takes half its relative error, and out two products more."""
    s = f64(s)
    D = s.shape[-1]
    w = f64(w) if w is not None else torch.ones(D, dtype=torch.float64)
    rstd = ((s * s).mean(-1) + eps) ** -0.5
    y = s * rstd[..., None] * w
    er = (0.5 * (D / 32 + 18) + 4) * U * rstd
    return (y, rstd), ((er / rstd)[..., None] * y.abs() + 3 * U * y.abs(), er)


def rms_bwd(dout, x, rstd, w, dres):
    """(dx, dweight) and bounds, for the given rstd."""
    x, r, dy = f64(x), f64(rstd)[..., None], f64(dout)
    D = x.shape[-1]
    w = f64(w) if w is not None else torch.ones(D, dtype=torch.float64)
    dr = f64(dres) if dres is not None else torch.zeros_like(x)
    xh, u = x * r, dy * w
    c = (u * xh).mean(-1, keepdim=True)
    n = D / 32 + 20
    ec = n * U * (u * xh).abs().mean(-1, keepdim=True)          # three roundings a term, those of the sum, the division's
    dx = r * (u - xh * c) + dr
    edx = r * (xh.abs() * ec + 4 * U * (u.abs() + (xh * c).abs())) + U * dx.abs()
    R = x.numel() // D
    flat = (dy * xh).reshape(-1, D)
    return (dx, flat.sum(0)), (edx, (R + 64) * U * flat.abs().sum(0))


def scales(y, block_rows):
    """Largest magnitude of each block of block_rows x 128, in 64 bits."""
    y = f64(y)
    R, D = y.shape
    p = torch.zeros(-(-R // block_rows) * block_rows, -(-D // 128) * 128, dtype=torch.float64)
    p[:R, :D] = y
    p = p.view(-1, block_rows, p.shape[1] // 128, 128)
    return p.abs().amax((1, 3))


def spread(c, R, D, block_rows):
    """The scales laid out for each value of [R, D]."""
    return f64(c).repeat_interleave(block_rows, 0)[:R].repeat_interleave(128, 1)[:, :D]


def check_e4m3(q, c, y, err, what):
    """q c is y (known to err) rounded to e4m3 in units of c: off by half a step at most, 2^-4 of the value, or 2^-10 c
    where e4m3 has no smaller exponent; beyond 448 c there is nothing, which err covers."""
    got = f64(q.float()) * c
    tol = torch.maximum((y.abs() + err) * 2.0 ** -4, c * 2.0 ** -10) + err
    assert torch.isfinite(got).all(), what
    worst = ((got - y).abs() / tol).max().item() if y.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its bound"


def fp8_linear(x, xs, w, ws):
    """out and bound.  Products of two e4m3 values are exact; a block's 128 terms and the blocks' sums are rounded, as
    are the scales' product and what it multiplies.  Twice that: a tensor core may cut instead of round."""
    (M, K), N = x.shape, w.shape[0]
    a = f64(x.float()) * spread(xs, M, K, 1)
    b = f64(w.float()) * spread(ws, N, K, 128)
    return a @ b.T, 2 * (128 + -(-K // 128) + 4) * U * (a.abs() @ b.abs().T)


def _logits(h, w):
    # fp32 sums of D products in any order, an accumulator that truncates counted double
    return h @ w.T, 2 * U * (h.shape[1] + 2) * (h.abs() @ w.abs().T)


def _kept(targets, V):
    t = targets.cpu().long()
    return t, (t >= 0) & (t < V)


def log_probs_fwd(h, w, targets, k):
    """(logp, entropy, lse, ids, top logps) and bounds; ids by the 64-bit logits, equal ones by the lower index."""
    h, w = f64(h), f64(w)
    V = w.shape[0]
    t, keep = _kept(targets, V)
    h = torch.where(keep[:, None], h, 0.0)
    l, el = _logits(h, w)
    el = el.max(-1, keepdim=True).values
    top = l.max(-1, keepdim=True).values
    lse = torch.logsumexp(l, -1, keepdim=True)
    lp = l - lse
    p, d = lp.exp(), l - top
    H = -(p * lp).sum(-1)
    # as the cross entropy's: the largest logit error, the sum's roundings, the logarithm's and the differences'
    e = (el + (V / 128 + 40) * U + 4 * U * (lse.abs() + l.abs().max(-1, keepdim=True).values))[:, 0]
    # entropy: an error of a logit counts p |log p + H|, that of an exponential's term (its argument's rounding, in units
    # of log2 e too, and the sums') once in log S and, times |d| + U / S, in U / S
    term = (V / 128 + 48) * U + 6 * U * d.abs()
    eH = (p * term * (1 + d.abs() + (p * d).sum(-1, keepdim=True).abs())).sum(-1) + \
        2 * (el * (p * (lp + H[:, None]).abs()).sum(-1, keepdim=True))[:, 0] + 6 * U * (H + (lse - top).abs()[:, 0])
    z = torch.zeros_like(H)
    v, ids = torch.sort(lp, dim=-1, descending=True, stable=True)
    rows = [torch.where(keep, x, z) for x in (lp.gather(1, t.clamp(0, V - 1)[:, None])[:, 0], H, lse[:, 0])]
    return (*rows, torch.where(keep[:, None], ids[:, :k], -1), torch.where(keep[:, None], v[:, :k], 0.0)), (2 * e, eH, e, 2 * e)


def log_probs_bwd(h, w, targets, lse, H, da, db, low_bits):
    """(dh, dweight) and bounds, for the given lse and H.  ``low_bits``: the logits' gradient enters the products rounded to
    bfloat16 in units of its row's weight, and dweight's other factor, that weight times h, is rounded too."""
    h, w, lse, da = f64(h), f64(w), f64(lse), f64(da)
    N, V = h.shape[0], w.shape[0]
    t, keep = _kept(targets, V)
    h = torch.where(keep[:, None], h, 0.0)
    a = torch.where(keep, da, 0.0)[:, None]
    b = torch.where(keep, f64(db), 0.0)[:, None] if db is not None else torch.zeros_like(a)
    H = torch.where(keep, f64(H), 0.0)[:, None] if db is not None else torch.zeros_like(a)
    lse = torch.where(keep, lse, 0.0)[:, None]
    l, el = _logits(h, w)
    lp = l - lse
    p = lp.exp()
    hot = torch.nn.functional.one_hot(t.clamp(0, V - 1), V).double()
    G = a * (hot - p) - b * p * (lp + H)
    ep = (el + 4 * U * (l.abs() + lse.abs()) + 4 * U) * 1.01          # relative, of p
    eG = p * (a.abs() * ep + b.abs() * (ep * (lp + H).abs() + el + 4 * U * (l.abs() + lse.abs() + H.abs())))
    eG = eG + 6 * U * (a.abs() * (hot + p) + b.abs() * p * (lp + H).abs())
    if low_bits:
        eG = eG + BF16 * G.abs()
    edh = eG @ w.abs() + 2 * U * (V + 64) * (G.abs() @ w.abs())
    edw = (eG + (BF16 if low_bits else 0.0) * G.abs()).T @ h.abs() + 2 * U * (N + 64) * (G.abs().T @ h.abs())
    return (G @ w, G.T @ h), (edh, edw)
