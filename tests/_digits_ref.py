"""Rows and weights that lay single digits of the linear of a few rows bare, and a model of its digits.

Each output multiplies one element of x alone, which lies far below the largest of its block of 16 and of its row; those
meet weights of zero.  So nothing of a sum's size hides an element's error, and the bound is the promised one: 2^-22 of the
block's largest or 2^-40 of the row's, and the output's rounding."""
import numpy as np
import torch

DEPTHS = (12, 13, 14, 15, 16, 17, 18, 19, 20)          # binades of the elements below their block's largest
BLOCKS = (0, 10, 0, 12, 15, 17, 0, 13, 16, 20, 11, 24)  # and of the blocks' largest below their row's


def make(rng, M, K):
    """bf16 x [M, K] and w [N, K], N = K / 16 * 9: output 9 b + j is the element j + 1 of block b."""
    nb = K // 16
    x = np.zeros((M, nb, 16))
    below = np.array([[BLOCKS[(b * 5 + m) % len(BLOCKS)] if b else 0 for b in range(nb)] for m in range(M)])
    top = np.exp2(-below + rng.integers(-20, 20, (M, 1)).astype(np.float64))
    x[:, :, 0] = top * rng.choice([-1.0, 1.0], (M, nb))
    for j, d in enumerate(DEPTHS):
        mantissa = rng.integers(128, 256, (M, nb)) | 1      # (the last bit set: all eight count)
        x[:, :, j + 1] = top * np.exp2(-d - 8.0) * mantissa * rng.choice([-1.0, 1.0], (M, nb))
    w = np.zeros((nb, len(DEPTHS), nb, 16))
    for b in range(nb):
        for j in range(len(DEPTHS)):
            w[b, j, b, j + 1] = rng.uniform(0.03, 0.06) * rng.choice([-1.0, 1.0])
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)  # noqa: E731
    x = bf(x.reshape(M, K))
    return x, bf(w.reshape(nb * len(DEPTHS), K))


def reference(x, w):
    """float64 (x w^T, the largest error): `w` float64 as it is held."""
    a = x.double()
    top = a.abs().unflatten(-1, (-1, 16)).amax(-1).repeat_interleave(16, -1)
    off = torch.maximum(2.0 ** -22 * top, 2.0 ** -40 * a.abs().amax(-1, keepdim=True))
    y = a @ w.T
    # (one product a sum: the fp32 steps behind it are three roundings)
    return y, 2.0 ** -8 * y.abs() + off @ w.abs().T * (1 + 2.0 ** -8) + 2.0 ** -22 * y.abs()


def digits(x, kept):
    """float64 of x as the kernel's digits have it: base 8, E2M1, f16 on the way; `kept`: which of the eight count."""
    values = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    mid, up = (values[1:] + values[:-1]) / 2, np.array([False, True] * 3 + [False])
    a = x.double().numpy().reshape(x.shape[0], -1, 16)
    exponent = lambda t: np.floor(np.log2(t)) - 1  # noqa: E731   the largest lies in [2, 4) of the unit
    e_row = exponent(np.abs(a).max((1, 2)))[:, None]
    below = np.minimum(17, e_row - exponent(np.abs(a).max(2)))
    unit = np.exp2(e_row - below)[..., None]
    left = (a / unit).astype(np.float16)
    got = np.zeros_like(a)
    for t in range(8):
        at = np.abs(left.astype(np.float64))[..., None]
        d = np.copysign(values[((at > mid) | ((at == mid) & up)).sum(-1)], left)
        if t in kept:
            got += d * 8.0 ** -t
        left = (8 * left.astype(np.float64) - 8 * d).astype(np.float16)
    return torch.from_numpy((got * unit).reshape(x.shape))
