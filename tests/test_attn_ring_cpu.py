"""The attention kernel's barriers, as modelled in attn_ring_model.py (CPU): no role goes on too early and none waits for
ever, in both kinds of units and both ring depths; with what the kernel must not do, the model fails."""
import os
import re

import pytest

from attn_ring_model import failures

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUNS = 400


def kernel():
    """Slots, places and stages as the kernel's source has them."""
    text = open(os.path.join(ROOT, "audio_dit_gb300", "csrc", "h3fp4_attn.cu")).read()
    number = lambda pattern: [int(x) for x in re.search(pattern, text).groups()]  # noqa: E731
    (masks,), (pieces,) = number(r"kMaskSlots = (\d+);"), number(r"kPieceSlots = (\d+);")
    q_solo, q_pair = number(r"kQ = kSolo \? (\d+) : (\d+);")
    all_tiles, width = number(r"kStages = \((\d+) - kQ\) \* \((\d+) / DP\);")
    assert re.search(r"q_full\[place % \(2 \* L::kQ\)\]", text) and re.search(r"kv_full\[place % \(2 \* kStages\)\]", text)
    return masks, pieces, {True: q_solo, False: q_pair}, all_tiles, width


def layout(solo, DP):
    masks, pieces, q, all_tiles, width = kernel()
    return dict(solo=solo, q_places=q[solo], stages=(all_tiles - q[solo]) * (width // DP), mask_slots=masks,
                piece_slots=pieces)


@pytest.mark.parametrize("DP", [64, 128])
@pytest.mark.parametrize("solo", [False, True])
def test_the_kernels_waits(solo, DP):
    assert failures(RUNS, **layout(solo, DP)) == {}


def test_one_full_barrier_per_stage_is_not_enough():
    """A role that waits for some of the ring's places only takes the fill before for its own."""
    broken = {}
    for solo in (False, True):
        for message, n in failures(RUNS, **layout(solo, 128), fulls=1).items():
            broken[message] = broken.get(message, 0) + n
    assert "wrong tile" in broken, broken


def test_fewer_mask_slots_than_the_ring_has_v_tiles_are_not_enough():
    assert failures(RUNS, **{**layout(True, 64), "mask_slots": 2}) != {}
