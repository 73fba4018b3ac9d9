"""The barriers of the one-kernel linear of a few rows, as modelled in rows_ring_model.py (CPU): no role goes on too early
and none waits for ever; with a ring whose slots go from warp to warp the model fails."""
import os
import re

from rows_ring_model import failures

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUNS = 300


FEW, MORE = (1, 2, 3, 4), (5, 6, 8)


def kernel():
    """Stages of the two forms, and how many stages' scales go together, as the kernel's source has them."""
    text = open(os.path.join(ROOT, "audio_dit_gb300", "csrc", "h3fp4_linear_rows.cu")).read()
    few, more = (int(n) for n in re.search(r"kStages = kRows == 4 \? (\d) : (\d);", text).groups())
    together = int(re.search(r"kTogether = (\d);", text).group(1))
    assert "every = 8 / row_warps, i0 = w / row_warps" in text
    assert "row_warps = kRows == 8 ? 8 : M > 2 ? 4 : M;" in text
    assert "1 + 4 + row_warps" in text and "mbar_init(&sf_full[i], 1 + row_warps)" in text
    return few, more, together


def test_the_kernels_waits():
    few, more, together = kernel()
    assert failures(RUNS, FEW, few, together) == {}
    assert failures(RUNS, MORE, more, together) == {}


def test_slots_have_to_be_one_warps():
    """A warp that skips fills of a slot takes one that is in use for free: seen as a launch failure with six stages."""
    assert failures(RUNS, FEW, 6, kernel()[2]) != {}
