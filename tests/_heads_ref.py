"""Plain 64-bit forms of the attention-side operators, and inputs for their tests."""
import math

import numpy as np
import torch


def norm_rope(x, w, cos, sin, pairs, off, eps):
    """float64 [M, H, D] of bf16 x; w fp32 [nseg, D] or None; cos/sin fp32 [M, rot/2] or None."""
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if w is not None:
        for i in range(len(off) - 1):
            y[off[i]:off[i + 1]] = y[off[i]:off[i + 1]] * w[i].double()
    if cos is not None:
        half = cos.shape[1]
        z = y.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            c, s = cos[:, i].double()[:, None], sin[:, i].double()[:, None]
            z[..., a] = y[..., a] * c - y[..., b] * s
            z[..., b] = y[..., b] * c + y[..., a] * s
        y = z
    return y


def attention(q, k, v, q_off, kv_off, scale, key_mask=None, k_ctx=None, v_ctx=None, ctx_mask=None):
    """float64 (out [M, Hq, D], lse [M, Hq], size [M, Hq, D], reach [M, Hq]).  ``size`` is sum_j p_j |v_j| / l, what
    the rounding errors of p scale with; ``reach`` is max_j scale sum_d |q_d k_jd|, what the error of a score scales
    with."""
    M, Hq, D = q.shape
    g = Hq // k.shape[1]
    out = torch.zeros(M, Hq, D, dtype=torch.float64)
    size = torch.zeros(M, Hq, D, dtype=torch.float64)
    reach = torch.zeros(M, Hq, dtype=torch.float64)
    lse = torch.full((M, Hq), -math.inf, dtype=torch.float64)
    for i in range(len(q_off) - 1):
        r = slice(q_off[i], q_off[i + 1])
        ki, vi = k[kv_off[i]:kv_off[i + 1]], v[kv_off[i]:kv_off[i + 1]]
        if key_mask is not None:
            on = key_mask[kv_off[i]:kv_off[i + 1]].bool()
            ki, vi = ki[on], vi[on]
        if k_ctx is not None:
            on = torch.ones(len(k_ctx), dtype=torch.bool) if ctx_mask is None else ctx_mask.bool()
            ki, vi = torch.cat([k_ctx[on], ki]), torch.cat([v_ctx[on], vi])
        if r.stop == r.start or len(ki) == 0:
            continue
        for h in range(Hq):
            z = q[r, h].double() @ ki[:, h // g].double().T * scale
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            n = p.sum(-1, keepdim=True)
            out[r, h] = p @ vi[:, h // g].double() / n
            size[r, h] = p @ vi[:, h // g].double().abs() / n
            lse[r, h] = (top + torch.log(n))[:, 0]
            reach[r, h] = (q[r, h].double().abs() @ ki[:, h // g].double().abs().T * scale).amax(-1)
    return out, lse, size, reach


def norm_rope_bound(ref, half, pairs):
    """|out - ref| of fp32 arithmetic and one rounding to bf16 (unit roundoff 2^-8).

    The sum of D <= 256 squares, the mean, rsqrt and three products are together within 2^-18 relative; a rotated
    element carries that of both elements of its pair, |a| + |b| <= sqrt(2) hypot(a', b')."""
    mag = ref.abs()
    if half:
        i = torch.arange(half)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        h = 1.5 * torch.hypot(mag[..., a], mag[..., b])
        mag = mag.clone()
        mag[..., a], mag[..., b] = h, h
    return 2.0 ** -8 * ref.abs() + 1.01 * 2.0 ** -18 * mag + 1e-38


def attention_bounds(out, lse, size, reach, D):
    """Bounds of |out - ref| and |lse - ref|.

    A score is a sum of D exact products in fp32, each of at most D + 8 steps off by 2^-23 of the sum of magnitudes;
    its error goes into p relatively, and once more through the sum l.  The p are rounded to bf16 (2^-8) for the
    product with V, the output once more (2^-8).  2^-11 covers the 2^x (2^-22), the scaled argument and sums of up to
    2^12 MMA steps (2^-24 each)."""
    z = reach * (D + 8) * 2.0 ** -23
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -11 + 4 * z)[..., None] * size + 1e-38
    return tol, 2.0 ** -11 + 2 * z + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


def rand_bf16(rng, *shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)) * scale).to(torch.bfloat16)


def lengths(rng, total, n):
    """n lengths that add up to total, some of them possibly zero."""
    cut = np.sort(rng.integers(0, total + 1, n - 1))
    return [0] + [int(c) for c in cut] + [total]
