"""The norm tests' comparison: a kernel that wrote NaN, left a place out or was off must not pass (CPU)."""
import numpy as np
import torch

import _heads_ref as R
from _norm_check import within


def test_what_must_fail():
    rng = np.random.default_rng(1)
    x = R.rand_bf16(rng, 9, 3, 64)
    ref = R.norm_rope(x, None, None, None, False, [0, 9], 1e-6)
    bound = R.norm_rope_bound(ref, 0, False)
    good = ref.to(torch.bfloat16)
    assert within(good, ref, bound)
    for bad in (torch.full_like(good, float("nan")), good.clone().index_put_((torch.tensor(4),), torch.tensor(float("nan")).bfloat16()),
                torch.zeros_like(good), good * 1.02):
        assert not within(bad, ref, bound)
