"""Plain 64-bit forms of a token's way through a block, and the bounds that their tests use."""
import torch


def block_norm(x, y, y_weight, gate, x_scale, weight, shift, scale, off, eps, post, layer):
    """float64 (out, x_out or None, tolerance of out, tolerance of x_out) of bf16 rows [M, K].

    Bounds.  A sum of K <= 32768 fp32 terms is taken as at most 32 additions in a thread and 10 over the threads: 2^-18
    of the sum of magnitudes covers it and the products around it.  An element of r is off by 2^-18 of |x_scale x| +
    |gate y'| (the sum of y^2 is in there), the mean by that of the mean magnitude; both reach z through rsqrt(var), once
    themselves and once through var (their root mean square, times z).  Each output is rounded to bf16 (2^-8)."""
    M, K = x.shape
    rows = lambda v: None if v is None else torch.cat(  # noqa: E731
        [v[i:i + 1].double().expand(off[i + 1] - off[i], -1) for i in range(len(off) - 1)])
    y_weight, gate, weight, shift, scale = (rows(v) for v in (y_weight, gate, weight, shift, scale))
    one = torch.ones(M, K, dtype=torch.float64)
    r, size, x_out, x_tol = x.double(), x.double().abs(), None, None
    if y is not None:
        b = y.double()
        if post:
            b = b / torch.sqrt((b * b).mean(-1, keepdim=True) + eps) * (one if y_weight is None else y_weight)
        b = b * (one if gate is None else gate)
        size = size * abs(x_scale) + b.abs()
        r = x_scale * r + b
        x_out, x_tol = r, 2.0 ** -8 * r.abs() + 2.0 ** -18 * size + 1e-38
    off_r = 2.0 ** -18 * size
    if layer:
        off_r = off_r + 2.0 ** -18 * r.abs().mean(-1, keepdim=True)
        r = r - r.mean(-1, keepdim=True)
    rs = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    z = r * rs
    off_z = rs * (off_r + z.abs() * off_r.pow(2).mean(-1, keepdim=True).sqrt()) + 2.0 ** -20 * z.abs()
    turn = (one if weight is None else weight) * (one if scale is None else 1 + scale)
    out = z * turn + (0 if shift is None else shift)
    tol = 2.0 ** -8 * out.abs() + 1.01 * off_z * turn.abs() + 1e-38
    if scale is not None:
        tol = tol + 2.0 ** -22 * (z * (one if weight is None else weight)).abs() * (1 + scale.abs())
    if shift is not None:
        tol = tol + 2.0 ** -22 * shift.abs()
    return out, x_out, tol, x_tol
