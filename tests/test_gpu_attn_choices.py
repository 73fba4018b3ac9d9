"""Attention (GPU) where units stay whole over several waves, and where a context walked
apart is joined row by row, against a plain 64-bit form."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import numpy as np  # noqa: E402

import _heads_ref as R  # noqa: E402
from test_gpu_attn import Case, built  # noqa: E402,F401


@pytest.mark.parametrize("M,T,Hq,Hkv,D", [(900, 300, 24, 24, 128), (2500, 300, 24, 24, 64), (513, 1100, 24, 8, 128),
                                          (1025, 900, 24, 24, 72), (700, 130, 40, 40, 8)])
def test_whole_units_of_one_segment(M, T, Hq, Hkv, D):
    Case(M, Hq, Hkv, D, [0, M], [0, T]).check()


@pytest.mark.parametrize("D", [64, 128])
def test_whole_units_of_ragged_segments(D):
    rng = np.random.default_rng(D)
    q_off, kv_off = R.lengths(rng, 1500, 7), R.lengths(rng, 2300, 7)
    c = Case(D, 12, 4, D, q_off, kv_off, ctx=77)
    c.key_mask = torch.from_numpy(rng.random(c.T) < 0.7)
    c.check()


@pytest.mark.parametrize("Hq,Hkv,D", [(7, 1, 128), (6, 2, 64), (4, 4, 40), (16, 4, 128), (130, 1, 16)])
@pytest.mark.parametrize("rows", [1, 3, 20])
def test_context_apart_joined_by_rows(Hq, Hkv, D, rows):
    """Blocks of the joining kernel hold rows of several segments and of two of the context's units."""
    n = 60 // rows + 7
    rng = np.random.default_rng(Hq + rows)
    q_off, kv_off = [0], [0]
    for i in range(n):  # some segments have no row, some no key of their own
        q_off.append(q_off[-1] + (0 if i % 7 == 3 else rows + i % 2))
        kv_off.append(kv_off[-1] + (0 if i % 5 == 2 else int(rng.integers(1, 150))))
    Case(rows, Hq, Hkv, D, q_off, kv_off, ctx=3001).check()


def test_context_apart_with_masks():
    n = 50
    q_off, kv_off = list(range(0, 2 * n + 1, 2)), list(range(0, 9 * n + 1, 9))
    c = Case(5, 8, 2, 128, q_off, kv_off, ctx=2500)
    c.ctx_mask = torch.from_numpy(np.arange(2500) % 3 != 1)
    c.key_mask = torch.from_numpy(np.arange(9 * n) // 9 % 4 != 0)   # every fourth segment's own keys are left out
    c.check()
    c.ctx_mask[:] = False                                           # then its rows have no key at all
    c.check()
