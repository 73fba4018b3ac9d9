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


# E2M1's magnitudes by code, and where one code ends and the next begins (a tie goes to the even code)
_E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def held(x, gscale):
    """float64 [..., H, D] of what bf16 rows are held as: blocks of 16 under the heads' global scales (fp32 [H]), each
    step of the format one fp32 operation (a sixth is a product with the rounded 1/6), and the bf16 that comes back."""
    s = gscale[:, None]
    b = x.float().unflatten(-1, (-1, 16))
    S = (b.abs().amax(-1) * torch.tensor(1.0 / 6.0) / s).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    eff = S * s
    r = torch.where(eff == 0, torch.zeros_like(eff), (1.0 / eff).clamp(max=torch.finfo(torch.float32).max))
    q = (b * r[..., None]).double()
    at = q.abs()[..., None]
    mid = (_E2M1[1:] + _E2M1[:-1]) / 2
    even_up = torch.tensor([False, True, False, True, False, True, False])   # the upper code is even: it takes the tie
    code = ((at > mid) | ((at == mid) & even_up)).sum(-1)
    v = torch.where(torch.signbit(q), -_E2M1[code], _E2M1[code]) * S.double()[..., None]
    return v.flatten(-2) * gscale.double()[:, None], (v.float() * s[..., None]).flatten(-2).to(torch.bfloat16)


def cache_attention(q, k, v, row_off, total, causal, scale, there=None):
    """float64 (out, lse, size, reach, keys) of rows q [M, Hq, D] over lists of each sequence's held keys and values
    [len, H, D]; `there`: per sequence a mask of positions whose page exists.  `size`, `reach` as in _heads_ref."""
    M, Hq, D = q.shape
    out, size = torch.zeros(M, Hq, D, dtype=torch.float64), torch.zeros(M, Hq, D, dtype=torch.float64)
    lse = torch.full((M, Hq), -float("inf"), dtype=torch.float64)
    reach, keys = torch.zeros(M, Hq, dtype=torch.float64), torch.zeros(M, dtype=torch.float64)
    for s, n in enumerate(total):
        g = Hq // k[s].shape[1]
        for r in range(row_off[s], row_off[s + 1]):
            last = n - (row_off[s + 1] - r) + 1 if causal else n
            on = torch.arange(len(k[s])) < last
            if there is not None:
                on &= there[s]
            keys[r] = int(on.sum())
            if not keys[r]:
                continue
            ki, vi = k[s][on].repeat_interleave(g, 1), v[s][on].repeat_interleave(g, 1)
            z = torch.einsum("hd,khd->hk", q[r].double(), ki) * scale
            lse[r] = torch.logsumexp(z, -1)
            p = torch.exp(z - lse[r][:, None])
            out[r] = torch.einsum("hk,khd->hd", p, vi)
            size[r] = torch.einsum("hk,khd->hd", p, vi.abs())
            reach[r] = (torch.einsum("hd,khd->hk", q[r].double().abs(), ki.abs()) * scale).amax(-1)
    return out, lse, size, reach, keys


def cache_attention_bounds(out, lse, size, reach, keys, top, D):
    """Bounds of |out - ref| and |lse - ref|; `top`: the largest |v|.

    A score is a sum of D exact products in fp32, each of at most D + 8 steps off by 2^-23 of the sum of magnitudes; its
    error goes into p relatively, and once more through the sum.  The p are rounded to fp16 (2^-11) for the product with
    V; those below 2^-25 vanish where the largest is 2^6 at least, so each key is off by 2^-31 of the largest value.  2^-11
    covers the 2^x (2^-22), its argument and sums of up to 2^13 fp32 steps (2^-24 each, twice).  bf16 outputs: 2^-8."""
    z = reach * (D + 8) * 2.0 ** -23
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2.0 ** -11 + 4 * z)[..., None] * size
    tol = tol + (keys * 2.0 ** -31 * top)[:, None, None] + 1e-38
    return tol, 2.0 ** -11 + 2 * z + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


def decode_weight(codes, sf, gscale, K):
    """float64 (W [N, K], the magnitudes) of NVFP4 codes, their 128x4-tiled block scales and the global scale."""
    N = codes.shape[0]
    values = torch.cat([_E2M1, -_E2M1])
    w = values[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    r, c = torch.arange(N)[:, None], torch.arange(K // 16)[None]
    at = ((r // 128) * (K // 64) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    S = sf.view(torch.float8_e4m3fn).double()[at]
    return w * S.repeat_interleave(16, 1) * float(gscale)


def linear_rows(x, w, bias, gate, resid, swiglu):
    """float64 (out, tolerance) of the linear of a few rows, with bounds in the manner of the linear's.

    A sum of K exact products is accumulated in fp32 (1e-5 of the sum of magnitudes, the linear's own), x enters with an
    error of at most 2^-22 of the largest of its block of 16; the output is rounded to bf16 once (2^-8)."""
    a = x.double()
    y, size = a @ w.T, a.abs() @ w.abs().T
    top = a.abs().unflatten(-1, (-1, 16)).amax(-1).repeat_interleave(16, -1)
    off = 1e-5 * size + 2.0 ** -22 * (top @ w.abs().T)
    if bias is not None:
        y = y + bias.double()
        off = off + 2.0 ** -22 * bias.double().abs()
    if swiglu:
        # the bf16 outputs g and u are off by their bounds; |silu'| <= 1.1; the fp32 evaluation 2^-17, h to bf16 2^-8
        tol = 2.0 ** -8 * y.abs() + off
        (g, u), (tg, tu) = (t.unflatten(-1, (-1, 2, 128)).unbind(-2) for t in (y, tol))
        g, u, tg, tu = (t.flatten(-2) if t.dim() > 2 else t for t in (g, u, tg, tu))
        s = g * torch.sigmoid(g)
        first = (s.abs() + 1.1 * tg) * tu + 1.1 * tg * u.abs()
        return s * u, first + (2.0 ** -8 + 2.0 ** -17) * ((s * u).abs() + first) + 1e-38
    if gate is not None:
        y, off = resid.double() + gate.double() * y, gate.double().abs() * off
        off = off + 2.0 ** -22 * (resid.double().abs() + y.abs())
    return y, 2.0 ** -8 * y.abs() + off + 1e-38
