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


def cache(pool=MB, n_pages=10, page=64, heads_=2, dim=64, table=2 * MB, max_pages=4, length=3 * MB, row_off=4 * MB,
          nseq=3, kg=None, vg=None):
    f = [pool or 0, n_pages, page, heads_, dim, table or 0, max_pages, length or 0, row_off or 0, nseq, kg or 0, vg or 0]
    return C.byref((C.c_int64 * 12)(*f))


def view(ptr=5 * MB, row=256, head=64):
    from audio_dit_gb300 import _Heads
    return C.byref(_Heads(ptr, row, head))


def rows_call(lib, fn="h3fp4_cache_append", k=None, v=None, M=3, **kw):
    return getattr(lib, fn)(k or view(), v or view(6 * MB), M, cache(**kw), None)


def attend(lib, q=None, M=3, Hq=4, scale=0.1, out=None, lse=None, flags=4096, ws=8 * MB, ws_bytes=1 << 40, **kw):
    return lib.h3fp4_cache_attn(q or view(), M, Hq, cache(**kw), scale, out or view(7 * MB), lse, flags, ws, ws_bytes, None)


def test_cache_refusals(lib):
    for call in (lambda **k: rows_call(lib, **k), lambda **k: rows_call(lib, "h3fp4_cache_read", **k),
                 lambda **k: attend(lib, **k)):
        for kw in (dict(dim=0), dict(dim=8), dict(dim=72), dict(dim=272), dict(heads_=0), dict(heads_=4097), dict(page=8),
                   dict(page=24), dict(page=1040), dict(nseq=0), dict(nseq=1025), dict(n_pages=0), dict(n_pages=1 << 31),
                   dict(max_pages=0), dict(max_pages=1 << 31), dict(M=-1), dict(M=(1 << 31) - 255)):
            assert call(**kw) == SHAPE, kw
        for kw in (dict(pool=None), dict(table=None), dict(length=None), dict(row_off=None, M=2)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(pool=MB + 8), dict(table=MB + 2), dict(length=MB + 1), dict(row_off=MB + 2), dict(kg=MB + 2),
                   dict(vg=MB + 3)):
            assert call(**kw) == ALIGN, kw
    for kw in (dict(k=view(0)), dict(v=view(0)), dict(fn="h3fp4_cache_read", k=view(0)),
               dict(fn="h3fp4_cache_read", v=view(5 * MB)), dict(fn="h3fp4_cache_read", k=view(row=64))):
        assert rows_call(lib, **kw) == INVALID, kw
    for kw in (dict(k=view(5 * MB + 2)), dict(v=view(row=4)), dict(v=view(head=-64))):
        assert rows_call(lib, **kw) == ALIGN, kw
    for kw in (dict(Hq=0), dict(Hq=3), dict(M=1 << 29)):
        assert attend(lib, **kw) == SHAPE, kw
    for kw in (dict(flags=1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
               dict(q=view(0)), dict(out=view(0)), dict(out=view()), dict(out=view(7 * MB, 64, 64)), dict(ws=None),
               dict(ws_bytes=1000)):
        assert attend(lib, **kw) == INVALID, kw
    for kw in (dict(q=view(5 * MB + 8)), dict(out=view(row=260)), dict(ws=8 * MB + 8), dict(lse=MB + 2)):
        assert attend(lib, **kw) == ALIGN, kw
    assert lib.h3fp4_cache_append(view(), view(), 3, None, None) == INVALID
    assert lib.h3fp4_selftest_cache_attn_timeout(None, 1, None) == INVALID
    assert lib.h3fp4_selftest_cache_attn_timeout(C.c_void_p(4104), 1, None) == ALIGN


def test_cache_sizes(lib):
    import torch

    import audio_dit_gb300 as A
    for heads_, D, page, width in ((2, 64, 16, 64), (1, 16, 32, 64), (8, 80, 64, 128), (3, 256, 1024, 256), (1, 144, 16, 256)):
        assert A.h3fp4_cache_page_bytes(heads_, D, page) == heads_ * page * width * 9 // 8
        c = A.alloc_kv_cache(5, heads_, D, page, device="cpu")
        assert c.numel() == 5 * A.h3fp4_cache_page_bytes(heads_, D, page)
    for bad in ((0, 64, 16), (1, 24, 16), (1, 64, 40), (1, 64, 2048), (1, 512, 16)):
        assert A.h3fp4_cache_page_bytes(*bad) == 0
        with pytest.raises(ValueError, match="refuse"):
            A.alloc_kv_cache(5, *bad, device="cpu")
    assert A.h3fp4_cache_attn_workspace_bytes(64) < A.h3fp4_cache_attn_workspace_bytes(256)
    assert A.h3fp4_cache_attn_workspace_bytes(40) == 0
    for bad in ((1, 1, 3, 2, 64), (1, 0, 2, 2, 64), (1, 1, 2, 2, 60)):
        with pytest.raises(ValueError, match="refuse"):
            A.alloc_cache_attn_workspace(*bad, device="cpu")
    x, t = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        A.h3fp4_cache_append(x, x, A.alloc_kv_cache(5, 2, 64, 16, device="cpu"), t, t[:, 0])


def rows(lib, x=MB, M=4, N=256, K=128, wc=2 * MB, wsf=3 * MB, wg=4 * MB, gate=None, stride=0, bias=None, resid=None,
         out=5 * MB, flags=0, ws=6 * MB, ws_bytes=1 << 40):
    return lib.h3fp4_linear_rows(x, M, N, K, wc, wsf, wg, gate, stride, bias, resid, out, flags, ws, ws_bytes, None)


def test_linear_rows_refusals(lib):
    G = dict(flags=4, gate=7 * MB, resid=8 * MB)
    for kw in (dict(M=0), dict(M=65), dict(M=-1), dict(N=0), dict(N=12), dict(N=(1 << 24) + 8), dict(K=0), dict(K=96),
               dict(K=(1 << 16) + 64), dict(flags=64, N=128)):
        assert rows(lib, **kw) == SHAPE, kw
    for kw in (dict(x=None), dict(wc=None), dict(wsf=None), dict(wg=None), dict(out=None), dict(ws=None), dict(ws_bytes=0),
               dict(flags=1), dict(flags=2), dict(bias=7 * MB), dict(gate=7 * MB), dict(flags=4), dict(flags=4, gate=7 * MB),
               dict(flags=4, resid=7 * MB), {**G, "flags": 68}, {**G, "stride": 255}, {**G, "stride": -1},
               {**G, "resid": 5 * MB + 16}, dict(out=MB), dict(out=MB + 1024 - 16), dict(out=MB - 2048 + 16),
               dict(out=2 * MB + 16384 - 16), dict(out=3 * MB + 2048 - 16), dict(flags=2, bias=5 * MB + 2048 - 16),
               {**G, "gate": 5 * MB + 2048 - 4}, {**G, "stride": 256, "gate": 5 * MB - 4096 + 4}, dict(out=6 * MB - 2048 + 16),
               dict(ws=MB + 1024 - 16), dict(ws=2 * MB + 16384 - 256), {**G, "resid": 6 * MB + 256}):
        assert rows(lib, **kw) == INVALID, kw
    for kw in (dict(x=MB + 2), dict(wc=2 * MB + 8), dict(wsf=3 * MB + 8), dict(wg=4 * MB + 2), dict(out=5 * MB + 4),
               dict(ws=6 * MB + 8), dict(flags=2, bias=7 * MB + 2), {**G, "gate": 7 * MB + 2}, {**G, "resid": 8 * MB + 8}):
        assert rows(lib, **kw) == ALIGN, kw


def test_linear_rows_python_checks(lib):
    import torch

    import audio_dit_gb300 as A
    assert lib.h3fp4_selftest_linear_rows_timeout(None, 1, None) == INVALID
    assert lib.h3fp4_selftest_linear_rows_timeout(C.c_void_p(4104), 1, None) == ALIGN
    assert (A.h3fp4_linear_rows_workspace_bytes(64, 128, 1024)
            >= A.h3fp4_linear_rows_workspace_bytes(9, 128, 256) + 128 * 128 + 9 * 256)   # what the self-test lays out
    assert A.ROWS_MAX == 64 and A.h3fp4_linear_rows_workspace_bytes(1, 8, 64) >= 256
    for bad in ((65, 8, 64), (0, 8, 64), (1, 4, 64), (1, 8, 32)):
        assert A.h3fp4_linear_rows_workspace_bytes(*bad) == 0
        with pytest.raises(ValueError, match="refuse"):
            A.alloc_rows_workspace(*bad, device="cpu")
    x, o = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 128, dtype=torch.bfloat16)
    codes, sf, g = torch.zeros(128, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.ones(1)
    with pytest.raises(ValueError, match="CUDA"):
        A.h3fp4_linear_rows(x, codes, sf, g, o, sf)
    with pytest.raises(ValueError, match="w_codes"):
        A.h3fp4_linear_rows(x, codes[:64], sf, g, o, sf)
    with pytest.raises(ValueError, match="w_sf"):
        A.h3fp4_linear_rows(x, codes, sf[:256], g, o, sf)
