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
