"""Segment tables of the attention side that are too short to hold a segment are refused (no GPU)."""
import ctypes as C

import pytest

from test_heads_cpu import SHAPE, lib, norm  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("table", [[], (), [0], (0,), [4]])
def test_short_tables(lib, table):  # noqa: F811
    import torch

    import audio_dit_gb300 as A
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: A.h3fp4_attn_workspace_bytes(4, 9, 2, 2, 64, table, table),
                 lambda: A.alloc_attn_workspace(4, 9, 2, 2, 64, table, table),
                 lambda: A.h3fp4_cross_attn(x, x, x, x, x, q_off=table, kv_off=table),
                 lambda: A.h3fp4_shared_attn(x, x, x, x, x, x, x, q_off=table, kv_off=table),
                 lambda: A.h3fp4_qk_norm_rope(x, None, x, None, seg_off=table)):
        with pytest.raises(ValueError, match="offset table"):
            call()


@pytest.mark.parametrize("nseg", [0, -1, -5])
def test_norm_table_without_a_segment(lib, nseg):  # noqa: F811
    """A table is read only as far as nseg says: one segment would be two entries of a table of one."""
    table = C.cast((C.c_int64 * 2)(0, 4), C.c_void_p)
    assert norm(lib, seg=table, nseg=nseg) == SHAPE
