"""64-bit plain forms of the gated scan, layer norm and linear cross entropy, on the CPU, and the error bounds that
their fp32 kernels are held to.  Nothing here is shared with the library.

Notation: u = 2^-24, the rounding of one fp32 operation.  A product of a chain of factors and a sum of n terms, each
rounded, is off by at most (number of roundings) u times the same expression with every term's magnitude, so each
bound is a count of roundings times a magnitude that is evaluated in 64 bits.
"""
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8 * 1.01   # one rounding to bfloat16 (8 significand bits), relative, with room for the fp32 error beneath it


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def bounds_of(x, cu):
    B, T = x.shape[0], x.shape[1]
    return [n * T for n in range(B + 1)] if cu is None else [int(v) for v in cu]


def scan_fwd(x, g, init, cu, gate):
    """(out, final, bound): bound is what an fp32 evaluation may be off by, for out and final alike the magnitude
    M_t = a M_{t-1} + hbar_t, hbar the scan of |c x|: a step multiplies what came before by a rounded exponential
    (2 u), a product of such factors (u) and an addition (u), and adds its own rounded input."""
    x, g = f64(x), f64(g)
    D = x.shape[-1]
    b = bounds_of(x, cu)
    fx, a = x.reshape(-1, D), g.reshape(-1, D).exp()
    c = -torch.expm1(g.reshape(-1, D)) if gate else torch.ones_like(a)
    N = len(b) - 1
    h0 = f64(init) if init is not None else torch.zeros(N, D, dtype=torch.float64)
    out, mag, final, fmag = torch.zeros_like(fx), torch.zeros_like(fx), h0.clone(), torch.zeros(N, D, dtype=torch.float64)
    for n in range(N):
        h, hb, m = h0[n], h0[n].abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(b[n], b[n + 1]):
            h = a[t] * h + c[t] * fx[t]
            hb = a[t] * hb + (c[t] * fx[t]).abs()
            m = a[t] * m + hb
            out[t], mag[t] = h, m
        final[n], fmag[n] = h, m
    return out.reshape(x.shape), final, 6 * U * mag.reshape(x.shape), 6 * U * fmag


def scan_bwd(x, g, out, dout, init, dfinal, cu, gate):
    """(dx, dg, dinit) and their bounds, counted as in scan_fwd with the products behind the scan."""
    g, out, dout = f64(g), f64(out), f64(dout)
    x = f64(x) if x is not None else torch.zeros_like(g)
    D = g.shape[-1]
    b = bounds_of(g, cu)
    N = len(b) - 1
    sh = g.shape
    g, x, out, dout = (t.reshape(-1, D) for t in (g, x, out, dout))
    a = g.exp()
    c = -torch.expm1(g) if gate else torch.ones_like(a)
    zero = torch.zeros(N, D, dtype=torch.float64)
    h0 = f64(init) if init is not None else zero
    e0 = f64(dfinal) if dfinal is not None else zero
    dx, dg, bx, bg = (torch.zeros_like(g) for _ in range(4))
    dinit, bi = e0.clone(), zero.clone()
    for n in range(N):
        e, eb, m = e0[n], e0[n].abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(b[n + 1] - 1, b[n] - 1, -1):
            prev = h0[n] if t == b[n] else out[t - 1]
            dh, hb = dout[t] + e, dout[t].abs() + eb
            dm = m + hb                      # of dH_t
            e, eb, m = a[t] * dh, a[t] * hb, a[t] * (dm + hb)
            dx[t], bx[t] = c[t] * dh, c[t].abs() * (dm + hb)
            dg[t] = e * (prev - x[t] if gate else prev)
            bg[t] = (m + eb) * (prev.abs() + (x[t].abs() if gate else 0))
        dinit[n], bi[n] = e, m
    return (dx.reshape(sh), dg.reshape(sh), dinit), (6 * U * bx.reshape(sh), 6 * U * bg.reshape(sh), 6 * U * bi)


def norm_fwd(x, w, b, eps):
    """(out, mean, rstd) and bounds.  A sum of D terms has at most n = D roundings on any path; the kernels' partial
    sums have far fewer (D / 32 + 16 covers a lane's share and the joining of 32 lanes and 16 parts)."""
    x = f64(x)
    D = x.shape[-1]
    n = D / 32 + 16
    mean = x.mean(-1)
    d = x - mean[..., None]
    var = (d * d).mean(-1)
    rstd = (var + eps) ** -0.5
    w = f64(w) if w is not None else torch.ones(D, dtype=torch.float64)
    b = f64(b) if b is not None else torch.zeros(D, dtype=torch.float64)
    y = d * rstd[..., None] * w + b
    em = n * U * x.abs().mean(-1)                              # the mean's
    ed = em[..., None] + 2 * U * (x.abs() + mean.abs()[..., None])   # a deviation's
    ev = (2 * d.abs() * ed + ed * ed).mean(-1) + n * U * var   # the variance's
    er = 0.5 * rstd ** 3 * ev + 4 * U * rstd                   # 1 / sqrt: first order in ev, and its own roundings
    ey = (rstd[..., None] * ed + er[..., None] * (d.abs() + ed)) * w.abs() + 4 * U * (y.abs() + b.abs())
    return (y, mean, rstd), (ey, em + U * mean.abs(), er)


def norm_bwd(dout, x, mean, rstd, w):
    dy, x, mean, rstd = f64(dout), f64(x), f64(mean)[..., None], f64(rstd)[..., None]
    D = x.shape[-1]
    w = f64(w) if w is not None else torch.ones(D, dtype=torch.float64)
    n = D / 32 + 20
    xh = (x - mean) * rstd
    u = dy * w
    c1, c2 = u.mean(-1, keepdim=True), (u * xh).mean(-1, keepdim=True)
    dx = rstd * (u - c1 - xh * c2)
    ex = 4 * U * rstd * (x.abs() + mean.abs())                 # xhat's
    e1 = n * U * u.abs().mean(-1, keepdim=True)
    e2 = (u.abs() * (ex + n * U * xh.abs())).mean(-1, keepdim=True)
    edx = rstd * (8 * U * (u.abs() + c1.abs() + (xh * c2).abs()) + e1 + xh.abs() * e2 + ex * (c2.abs() + e2))
    rows = dy.reshape(-1, D).shape[0]
    m = rows / 16 + 64                                         # roundings on the longest path of a column's sum
    flat = lambda t: t.reshape(-1, D)  # noqa: E731
    dw, db = flat(dy * xh).sum(0), flat(dy).sum(0)
    edw = flat(dy.abs() * (ex + m * U * xh.abs())).sum(0)
    edb = m * U * flat(dy.abs()).sum(0)
    return (dx, dw, db), (edx, edw, edb)


def _logits(h, w):
    D = h.shape[1]
    # fp32 sums of D products in any order, an accumulator that truncates counted double
    return h @ w.T, 2 * U * (D + 2) * (h.abs() @ w.abs().T)


def ce_fwd(h, w, targets):
    h, w, t = f64(h), f64(w), targets.cpu().long()
    V = w.shape[0]
    keep = (t >= 0) & (t < V)
    h = torch.where(keep[:, None], h, 0.0)
    l, el = _logits(h, w)
    lse = torch.logsumexp(l, -1)
    at = l.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    # lse moves by no more than the largest logit error; the sum and its exponentials add a relative error of
    # (V / 128 + 40) u to the sum, an absolute one to its logarithm
    e = el.max(-1).values + (V / 128 + 40) * U + 4 * U * (lse.abs() + l.abs().max(-1).values)
    z = torch.zeros_like(lse)
    return (torch.where(keep, lse - at, z), torch.where(keep, lse, z)), (2 * e, e)


def ce_bwd(h, w, targets, lse, dloss, low_bits):
    """(dh, dweight) and bounds.  ``low_bits``: softmax - onehot enters the products rounded to bfloat16, and dweight's
    other factor, dloss h in units of the largest dloss, is rounded too."""
    h, w, t, lse, dl = f64(h), f64(w), targets.cpu().long(), f64(lse), f64(dloss)
    N, V, D = h.shape[0], w.shape[0], h.shape[1]
    keep = (t >= 0) & (t < V)
    h = torch.where(keep[:, None], h, 0.0)
    dl = torch.where(keep, dl, 0.0)
    lse = torch.where(keep, lse, 0.0)
    l, el = _logits(h, w)
    p = torch.exp(l - lse[:, None])
    hot = torch.nn.functional.one_hot(t.clamp(0, V - 1), V).double()
    G = (p - hot) * dl[:, None]
    # exp's argument is off by el and its own rounding; then three roundings, and one to bfloat16
    eG = dl.abs()[:, None] * p * (el + 4 * U * (l.abs() + lse.abs()[:, None]) + 4 * U) * 1.01 + 4 * U * G.abs()
    if low_bits:
        eG = eG + BF16 * G.abs()
    edh = eG @ w.abs() + 2 * U * (V + 64) * (G.abs() @ w.abs())
    edw = (eG + (BF16 if low_bits else 0.0) * G.abs()).T @ h.abs() + 2 * U * (N + 64) * (G.abs().T @ h.abs())
    return (G @ w, G.T @ h), (edh, edw)


def check(got, ref, bound, what):
    """Elementwise: within the bound, and one rounding where the result is bfloat16."""
    g = f64(got)
    assert tuple(g.shape) == tuple(ref.shape), f"{what}: shape {tuple(g.shape)} instead of {tuple(ref.shape)}"
    tol = bound + 1e-37
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + BF16) + BF16 * ref.abs()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    worst = ((g - ref).abs() / tol).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its bound (largest difference {(g - ref).abs().max().item():.3g})"
