"""Segment tables of the linear's calls that are too short to hold a segment are refused before the library reads
them (no GPU)."""
import pytest


@pytest.mark.parametrize("table", [[], (), [0], (0,), [4]])
def test_short_tables(table):
    import torch

    import audio_dit_gb300 as A
    from audio_dit_gb300 import build
    build.build()
    x, b, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.uint8), torch.zeros(1)
    for call in (lambda: A.h3fp4_linear(x, b, b, f, x, b, seg_off=table),
                 lambda: A.h3fp4_quantize_act(x, b, b, f, b, seg_off=table)):
        with pytest.raises(ValueError, match="offset table"):
            call()
