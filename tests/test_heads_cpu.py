"""Host-side checks of the attention-side entry points (no GPU): what they refuse, and their workspace sizes."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from audio_dit_gb300 import build
    build.build()
    import audio_dit_gb300 as A
    return A.load_library()


def heads(ptr=1 << 20, row=256, head=128):
    from audio_dit_gb300 import _Heads
    return C.byref(_Heads(ptr, row, head))


OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
P = C.c_void_p(4096)


def norm(lib, q=None, k=None, M=4, Hq=2, Hk=2, D=128, qw=None, kw=None, cos=None, sin=None, rot=0, seg=None, nseg=1,
         eps=1e-6, qo=None, ko=None, flags=0):
    return lib.h3fp4_qk_norm_rope(q or heads(), k, M, Hq, Hk, D, qw, kw, cos, sin, rot, seg, nseg, eps,
                                  qo or heads(2 << 20), ko, flags, None)


def test_norm_rope_refusals(lib):
    for kw in (dict(D=4), dict(D=12), dict(D=264), dict(M=-1), dict(M=1 << 31), dict(Hq=0), dict(rot=8, cos=P, sin=P),
               dict(rot=144, cos=P, sin=P), dict(rot=-16), dict(k=heads(3 << 20), ko=heads(4 << 20), Hk=0),
               dict(seg=C.cast((C.c_int64 * 10)(*range(9), 4), C.c_void_p), nseg=9)):
        assert norm(lib, **kw) == SHAPE, kw
    for kw in (dict(q=heads(0)), dict(qo=heads(0)), dict(k=heads(3 << 20)), dict(ko=heads(3 << 20)), dict(flags=1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rot=16), dict(rot=16, cos=P),
               dict(qo=heads(1 << 20, 512)),                       # another view of the same start
               dict(qo=heads(2 << 20, 256, 64)),                   # heads of the output overlap
               dict(qo=heads(2 << 20, 128, 128)),                  # rows of the output overlap
               dict(k=heads(2 << 20), ko=heads(4 << 20)), dict(k=heads(3 << 20), ko=heads(2 << 20)),
               dict(k=heads(3 << 20), ko=heads(1 << 20)),
               dict(seg=C.cast((C.c_int64 * 3)(0, 2, 5), C.c_void_p), nseg=2)):
        assert norm(lib, **kw) == INVALID, kw
    odd = C.c_void_p(4100)
    for kw in (dict(q=heads((1 << 20) + 2)), dict(q=heads(row=260)), dict(q=heads(head=4)), dict(q=heads(row=0)),
               dict(q=heads(head=-128)), dict(qo=heads((2 << 20) + 8)), dict(qw=odd),
               dict(rot=16, cos=odd, sin=P), dict(rot=16, cos=P, sin=odd)):
        assert norm(lib, **kw) == ALIGN, kw


def attn(lib, q=None, k=None, v=None, kc=None, vc=None, M=4, T=9, ctx=0, Hq=2, Hkv=2, D=128, q_off=None, kv_off=None,
         nseg=1, scale=0.1, out=None, lse=None, ws=P, ws_bytes=1 << 40):
    t = lambda x: None if x is None else C.cast((C.c_int64 * len(x))(*x), C.c_void_p)  # noqa: E731
    args = (M, T, ctx) if ctx else (M, T)
    a = [q or heads(), k or heads(2 << 20), v or heads(3 << 20)]
    o = out or heads(6 << 20)
    if ctx:
        return lib.h3fp4_shared_attn(*a, kc, vc, *args, Hq, Hkv, D, t(q_off), t(kv_off), nseg, None, None, scale, o,
                                     lse, ws, ws_bytes, None)
    return lib.h3fp4_cross_attn(*a, *args, Hq, Hkv, D, t(q_off), t(kv_off), nseg, None, scale, o, lse, ws, ws_bytes,
                                None)


def test_attention_refusals(lib):
    for kw in (dict(D=4), dict(D=20), dict(D=136), dict(Hq=3), dict(Hq=0), dict(Hkv=0), dict(M=-1), dict(T=-1),
               dict(M=1 << 31), dict(T=1 << 31), dict(T=(1 << 31) - 255), dict(M=1 << 30, Hq=2),
               dict(M=1 << 26, T=(1 << 31) - 256), dict(q_off=[0] * 257 + [4], kv_off=[0] * 257 + [9], nseg=257),
               dict(q_off=[0, 4], kv_off=[0, 9], nseg=0)):
        assert attn(lib, **kw) == SHAPE, kw
    for kw in (dict(q_off=[0, 4]), dict(kv_off=[0, 9]), dict(nseg=2), dict(q_off=[0, 3], kv_off=[0, 9]),
               dict(q_off=[1, 4], kv_off=[0, 9]), dict(q_off=[0, 3, 2, 4], kv_off=[0, 3, 3, 9], nseg=3),
               dict(q_off=[0, 4], kv_off=[0, 8]), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q=heads(0)), dict(k=heads(0)), dict(out=heads(0)), dict(ws=None),
               dict(ws_bytes=255), dict(out=heads(1 << 20)), dict(out=heads(2 << 20)), dict(out=heads(3 << 20)),
               dict(out=heads(6 << 20, 128, 128)), dict(ctx=5, kc=heads(4 << 20)),
               dict(ctx=5, kc=heads(4 << 20), vc=heads(6 << 20))):
        assert attn(lib, **kw) == INVALID, kw
    for kw in (dict(q=heads((1 << 20) + 8)), dict(k=heads(row=132)), dict(v=heads(head=2)), dict(out=heads((6 << 20) + 2)),
               dict(ws=C.c_void_p(4104)), dict(lse=C.c_void_p(4097)),
               dict(ctx=5, kc=heads((4 << 20) + 2), vc=heads(5 << 20))):
        assert attn(lib, **kw) == ALIGN, kw


def test_selftest_refusals(lib):
    assert lib.h3fp4_selftest_attn_timeout(None, 1, None) == INVALID
    assert lib.h3fp4_selftest_attn_timeout(C.c_void_p(4104), 1, None) == ALIGN


def test_workspace_bytes(lib):
    import audio_dit_gb300 as A
    assert A.h3fp4_attn_workspace_bytes(0, 0, 2, 2, 64) >= 256
    assert A.h3fp4_attn_workspace_bytes(100, 100, 2, 2, 64) >= 256
    for bad in ((10, 10, 3, 2, 64), (10, 10, 2, 2, 65), (-1, 10, 2, 2, 64)):
        assert A.h3fp4_attn_workspace_bytes(*bad) == 0
    assert A.h3fp4_attn_workspace_bytes(10, 10, 2, 2, 64, [0, 4, 10], [0, 9, 10]) >= 256
    assert A.h3fp4_attn_workspace_bytes(10, 10, 2, 2, 64, [0, 4, 9], [0, 9, 10]) == 0


def test_python_checks(lib):
    import torch

    import audio_dit_gb300 as A
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        A.h3fp4_qk_norm_rope(x, None, x, None)
    with pytest.raises(ValueError, match="go together"):
        A.h3fp4_qk_norm_rope(x, x, x, None)
    with pytest.raises(ValueError, match="go together"):
        A.h3fp4_cross_attn(x, x, x, x, x, q_off=[0, 4])
    with pytest.raises(ValueError, match="same length"):
        A.h3fp4_cross_attn(x, x, x, x, x, q_off=[0, 4], kv_off=[0, 1, 4])
    with pytest.raises(ValueError, match="refuse"):
        A.alloc_attn_workspace(4, 4, 3, 2, 64)
