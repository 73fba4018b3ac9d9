"""The checks of _attn_counts.py on a plain fp32 form with the kernels' roundings (CPU): they pass it, and fail the same
with one key lost or counted twice."""
import math

import numpy as np
import pytest
import torch

import _attn_counts as N
import _heads_ref as R


def plain(q, k, v, scale, extra=None):
    """fp32 softmax, weights rounded to bf16 for their product with V; ``extra``: how often each key counts."""
    w = torch.ones(k.shape[0]) if extra is None else extra
    out, lse = torch.empty(q.shape), torch.empty(q.shape[:2])
    for h in range(q.shape[1]):
        z = q[:, h].float() @ k[:, h].float().T * scale
        top = z.amax(-1, keepdim=True)
        p = torch.exp(z - top) * w
        n = p.sum(-1, keepdim=True)
        out[:, h] = p.to(torch.bfloat16).float() @ v[:, h].float() / n
        lse[:, h] = (top + torch.log(n))[:, 0]
    return out.to(torch.bfloat16), lse


@pytest.mark.parametrize("T,D", [(6001, 128), (30001, 64), (70000, 128)])
def test_counting(T, D):
    q, k = torch.zeros(3, 1, D, dtype=torch.bfloat16), torch.ones(T, 1, D, dtype=torch.bfloat16)
    every = N.period(T, D)
    share, total = N.counts([0, 3], [0, T], 0, D, every, 0)
    v = N.marked(0, T, 1, D, every, 0)
    assert N.counted(*plain(q, k, v, 0.1), [0, 3], share, total) is None
    for key in (5, T // 2 // every * every, T // every * every - every + 7):
        for times in (0.0, 2.0):
            w = torch.ones(T)
            w[key] = times
            assert N.counted(*plain(q, k, v, 0.1, w), [0, 3], share, total) is not None
    # in the sums alone, or in the products alone
    w = torch.ones(T)
    w[every + 3] = 0.0
    out, lse = plain(q, k, v, 0.1)
    bad_out, bad_lse = plain(q, k, v, 0.1, w)
    assert N.counted(out, bad_lse, [0, 3], share, total) and N.counted(bad_out, lse, [0, 3], share, total)


@pytest.mark.parametrize("T,D", [(6001, 128), (20001, 64)])
def test_norms(T, D):
    rng = np.random.default_rng(T)
    q, k, v = (R.rand_bf16(rng, n, 1, D) for n in (8, T, T))
    scale = 0.3 * D ** -0.5      # weights of like size: no key is too small to be missed
    ref = R.attention(q, k, v, [0, 8], [0, T], scale)[0]
    assert N.far_off(plain(q, k, v, scale)[0], ref) is None
    for times in (0.0, 2.0):
        w = torch.ones(T)
        w[T // 3] = times
        assert N.far_off(plain(q, k, v, scale, w)[0], ref) is not None


def test_no_key():
    share, total = N.counts([0, 2, 4], [0, 0, 5], 0, 8, 8, 0)
    assert list(total) == [0, 5]
    out, lse = torch.zeros(4, 1, 8), torch.full((4, 1), -math.inf)
    out[2:] = torch.from_numpy(share[1] / 5).to(torch.bfloat16).float()
    lse[2:] = math.log(5)
    assert N.counted(out, lse, [0, 2, 4], share, total) is None
    out[0, 0, 0] = 1.0
    assert N.counted(out, lse, [0, 2, 4], share, total) == "segment 0 has no key"
