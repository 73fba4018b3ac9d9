"""Host-side checks of a token's way through a block (no GPU): what the entry points refuse."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from audio_dit_gb300 import build
    build.build()
    import audio_dit_gb300 as A
    return A.load_library()


OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
MB = 1 << 20


def norm(lib, x=MB, y=2 * MB, M=4, K=64, yw=None, gate=None, xs=1.0, w=None, shift=None, scale=None, seg=None, nseg=1,
         eps=1e-6, xo=3 * MB, out=4 * MB, amax=None, flags=0):
    t = None if seg is None else C.cast((C.c_int64 * len(seg))(*seg), C.c_void_p)
    return lib.h3fp4_block_norm(x, y, M, K, yw, gate, xs, w, shift, scale, t, nseg, eps, xo, out, amax, flags, None)


def test_block_norm_refusals(lib):
    inf, nan = float("inf"), float("nan")
    for kw in (dict(K=0), dict(K=4), dict(K=12), dict(K=32776), dict(M=-1), dict(M=1 << 31),
               dict(seg=[0] * 9 + [4], nseg=9)):
        assert norm(lib, **kw) == SHAPE, kw
    for kw in (dict(flags=1), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(xs=nan), dict(xs=inf), dict(x=None),
               dict(out=None, xo=None), dict(out=None, w=MB), dict(out=None, shift=MB), dict(out=None, scale=MB),
               dict(out=None, amax=MB), dict(out=None, flags=2048), dict(y=None), dict(y=None, xo=None, gate=MB),
               dict(y=None, xo=None, flags=1024), dict(y=None, xo=None, yw=MB), dict(yw=MB), dict(seg=[0, 3], nseg=1),
               dict(seg=[0, 3, 2, 4], nseg=3), dict(nseg=2), dict(out=3 * MB), dict(out=3 * MB + 16),
               dict(xo=MB + 512 - 16), dict(xo=MB - 512 + 16), dict(out=2 * MB + 16)):
        assert norm(lib, **kw) == INVALID, kw
    for kw in (dict(x=MB + 2), dict(y=MB + 8), dict(xo=3 * MB + 4), dict(out=4 * MB + 8), dict(gate=MB + 4),
               dict(w=MB + 8), dict(shift=MB + 4), dict(scale=MB + 4), dict(yw=MB + 4, flags=1024), dict(amax=MB + 2)):
        assert norm(lib, **kw) == ALIGN, kw


def test_block_norm_python_checks(lib):
    import torch

    import audio_dit_gb300 as A
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        A.h3fp4_block_norm(x, x)
    with pytest.raises(TypeError, match="Tensor"):
        A._bf16(3, "x", (4, 64))
    with pytest.raises(ValueError, match="two entries"):
        A.h3fp4_block_norm(x, x, seg_off=[4])
