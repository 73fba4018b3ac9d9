"""Outputs of the norms and of the linear of a few rows over the vectors that they read (no GPU: only calls that are refused
are made)."""
import ctypes as C

import pytest

INVALID, MB = 1, 1 << 20


@pytest.fixture(scope="module")
def lib():
    from audio_dit_gb300 import build
    build.build()
    import audio_dit_gb300 as A
    return A.load_library()


def norm(lib, yw=None, gate=None, w=None, shift=None, scale=None, amax=None):
    # 4 rows of 64 (512 bytes) in two segments (vectors of 512 bytes): x, y, x_out, out at 1, 2, 3, 4 MB
    off = C.cast((C.c_int64 * 3)(0, 1, 4), C.c_void_p)
    return lib.h3fp4_block_norm(MB, 2 * MB, 4, 64, yw, gate, 1.0, w, shift, scale, off, 2, 1e-6, 3 * MB, 4 * MB, amax, 1024,
                                None)


@pytest.mark.parametrize("vector", ["yw", "gate", "w", "shift", "scale"])
def test_block_norm(lib, vector):
    for out in (3 * MB, 4 * MB):
        for at in (out, out + 512 - 16, out - 512 + 16):
            assert norm(lib, **{vector: at}) == INVALID, at - out
    for at in (5 * MB, 5 * MB + 512 - 4):
        assert norm(lib, **{vector: 5 * MB}, amax=at) == INVALID, at
    for at in (MB + 4, 2 * MB + 508, 3 * MB, 4 * MB + 8):
        assert norm(lib, amax=at) == INVALID, at


def test_linear_rows(lib):
    def rows(wg, out=5 * MB, ws=6 * MB):
        return lib.h3fp4_linear_rows(MB, 4, 256, 128, 2 * MB, 3 * MB, wg, None, 0, None, None, out, 0, ws, 1 << 40, None)
    assert rows(5 * MB) == INVALID and rows(5 * MB + 4 * 512 - 4) == INVALID and rows(6 * MB + 1024) == INVALID
