"""The barriers of the one-kernel linear of a few rows, as modelled in rows_ring_model.py (CPU): no role goes on too early
and none waits for ever; with a ring whose slots go from warp to warp the model fails."""
import os
import re

from rows_ring_model import failures

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUNS = 300


def kernel():
    """Stages, and how many stages' scales go together, as the kernel's source has them."""
    text = open(os.path.join(ROOT, "audio_dit_gb300", "csrc", "h3fp4_linear_rows.cu")).read()
    stages = int(re.search(r"kFewStages = (\d);", text).group(1))
    together = int(re.search(r"kTogether = (\d);", text).group(1))
    assert "every = 8 / row_warps, i0 = w / row_warps" in text
    assert "row_warps = M > 2 ? 4 : M;" in text
    assert "1 + 4 + row_warps" in text and "mbar_init(&sf_full[i], 1 + row_warps)" in text
    return stages, together


def test_the_kernels_waits():
    assert failures(RUNS, *kernel()) == {}


def test_slots_have_to_be_one_warps():
    """A warp that skips fills of a slot takes one that is in use for free: seen as a launch failure with six stages."""
    assert failures(RUNS, 6, kernel()[1]) != {}
