"""audio_dit_gb300 -- GB300 (sm_103a) NVFP4 linear path of a joint video/audio DiT.

Thin Python binding over the C ABI in ``include/h3fp4.h`` (``libh3fp4.so``):
the functions below carry the C names and only marshal arguments -- every
step of the path (modulation, amax, block scales, E2M1 packing, block-scaled
GEMM, bias/gate/residual epilogue) runs in the library's CUDA kernels.
PyTorch supplies device memory and streams.  There is no CPU or eager
fallback: if the library is missing or the device is not sm_103 the calls
raise.
"""
from __future__ import annotations

import ctypes as C
import os
from array import array
from typing import Optional, Sequence

import torch

__all__ = [
    "H3FP4Error", "PROLOGUE_MOD", "EPI_BIAS", "EPI_GATE_RESID", "GSCALE_GIVEN", "A_PREQUANT",
    "EPI_SWIGLU", "EPI_AMAX", "FUSED_QUANT", "h3fp4_ws_out_amax", "h3fp4_selftest_pack_timeout",
    "MAX_SEGMENTS", "library_path", "load_library", "h3fp4_codes_bytes", "h3fp4_sf_bytes",
    "h3fp4_workspace_bytes", "h3fp4_quantize_weight", "h3fp4_quantize_act", "h3fp4_linear",
    "h3fp4_check", "h3fp4_act_amax", "h3fp4_gscale_from_amax", "h3fp4_selftest_timeout", "h3fp4_measure_fp4_peak", "h3fp4_measure_fp4_pair_peak", "h3fp4_measure_fp4_form", "MMA_FORMS", "h3fp4_quantize_act_noalloc",
    "h3fp4_linear_swiglu_nvfp4", "h3fp4_qk_norm_rope", "h3fp4_cross_attn", "h3fp4_shared_attn",
    "h3fp4_attn_workspace_bytes", "alloc_attn_workspace", "h3fp4_selftest_attn_timeout", "ROPE_PAIRS", "ATTN_MAX_SEGMENTS",
    "h3fp4_set_wait_limit_ns", "h3fp4_status_string", "alloc_nvfp4", "alloc_workspace",
    "h3fp4_block_norm", "NORM_POST", "NORM_LAYER", "CAUSAL", "h3fp4_cache_append", "h3fp4_cache_read",
    "h3fp4_cache_attn", "h3fp4_cache_page_bytes", "h3fp4_cache_attn_workspace_bytes", "alloc_kv_cache",
    "alloc_cache_attn_workspace", "h3fp4_linear_rows",
    "h3fp4_linear_rows_workspace_bytes", "alloc_rows_workspace", "ROWS_MAX", "h3fp4_selftest_cache_attn_timeout",
    "h3fp4_selftest_linear_rows_timeout",
]

PROLOGUE_MOD = 1
EPI_BIAS = 2
EPI_GATE_RESID = 4
GSCALE_GIVEN = 16
A_PREQUANT = 32
EPI_SWIGLU = 64
EPI_AMAX = 128
FUSED_QUANT = 256
ROPE_PAIRS = 512
NORM_POST = 1024
NORM_LAYER = 2048
CAUSAL = 4096
MAX_SEGMENTS = 8
ATTN_MAX_SEGMENTS = 256
ROWS_MAX = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


class H3FP4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: h3fp4 status {status} ({h3fp4_status_string(status)})")


class _Heads(C.Structure):
    """h3fp4_heads: a strided bf16 [rows][heads][D] tensor."""
    _fields_ = [("ptr", C.c_void_p), ("row_stride", C.c_int64), ("head_stride", C.c_int64)]


def library_path() -> str:
    return os.path.join(_HERE, "_build", "libh3fp4.so")


def load_library():
    """Load libh3fp4.so (build it first with ``python -m audio_dit_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"libh3fp4.so not built ({path}); run `python -m audio_dit_gb300.build`")
    L = C.CDLL(path)
    i64, vp, i32, sz, hp = C.c_int64, C.c_void_p, C.c_int, C.c_size_t, C.c_void_p  # hp: h3fp4_heads
    sig = {
        "h3fp4_codes_bytes": (sz, [i64, i64]),
        "h3fp4_sf_bytes": (sz, [i64, i64]),
        "h3fp4_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "h3fp4_quantize_weight": (i32, [vp, i64, i64, vp, vp, vp, vp, vp]),
        "h3fp4_quantize_act": (i32, [vp, i64, i64, vp, vp, vp, i32, vp, vp, vp, i32, vp, vp]),
        "h3fp4_linear": (i32, [vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp,
                               i32, vp, vp]),
        "h3fp4_act_amax": (i32, [vp, i64, i64, vp, vp, vp, i32, vp, i32, vp, vp]),
        "h3fp4_linear_swiglu_nvfp4": (i32, [vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp,
                                            i32, vp, vp]),
        "h3fp4_gscale_from_amax": (i32, [vp, vp, vp]),
        "h3fp4_ws_out_amax": (vp, [vp]),
        "h3fp4_selftest_timeout": (i32, [vp, C.c_uint64, vp]),
        "h3fp4_selftest_pack_timeout": (i32, [vp, vp, vp, C.c_uint64, vp]),
        "h3fp4_measure_fp4_peak": (i32, [i32, vp, vp]),
        "h3fp4_measure_fp4_pair_peak": (i32, [i32, vp, vp]),
        "h3fp4_measure_fp4_form": (i32, [i32, i32, vp, vp]),
        "h3fp4_quantize_act_noalloc": (i32, [vp, i64, i64, vp, vp, vp, i32, vp, vp, vp, i32, vp]),
        "h3fp4_qk_norm_rope": (i32, [hp, hp, i64, i32, i32, i32, vp, vp, vp, vp, i32, vp, i32, C.c_float, hp, hp, i32,
                                     vp]),
        "h3fp4_cross_attn": (i32, [hp, hp, hp, i64, i64, i32, i32, i32, vp, vp, i32, vp, C.c_float, hp, vp, vp, sz,
                                   vp]),
        "h3fp4_shared_attn": (i32, [hp, hp, hp, hp, hp, i64, i64, i64, i32, i32, i32, vp, vp, i32, vp, vp, C.c_float,
                                    hp, vp, vp, sz, vp]),
        "h3fp4_attn_workspace_bytes": (sz, [i64, i64, i64, i32, i32, i32, vp, vp, i32]),
        "h3fp4_selftest_attn_timeout": (i32, [vp, C.c_uint64, vp]),
        "h3fp4_block_norm": (i32, [vp, vp, i64, i64, vp, vp, C.c_float, vp, vp, vp, vp, i32, C.c_float, vp, vp, vp, i32,
                                   vp]),
        "h3fp4_linear_rows": (i32, [vp, i64, i64, i64, vp, vp, vp, vp, i64, vp, vp, vp, i32, vp, sz, vp]),
        "h3fp4_linear_rows_workspace_bytes": (sz, [i64, i64, i64]),
        "h3fp4_selftest_linear_rows_timeout": (i32, [vp, C.c_uint64, vp]),
        "h3fp4_cache_page_bytes": (sz, [i32, i32, i32]),
        "h3fp4_cache_append": (i32, [hp, hp, i64, vp, vp]),
        "h3fp4_cache_read": (i32, [hp, hp, i64, vp, vp]),
        "h3fp4_cache_attn": (i32, [hp, i64, i32, vp, C.c_float, hp, vp, i32, vp, sz, vp]),
        "h3fp4_cache_attn_workspace_bytes": (sz, [i32]),
        "h3fp4_selftest_cache_attn_timeout": (i32, [vp, C.c_uint64, vp]),
        "h3fp4_check": (i32, [vp, vp]),
        "h3fp4_set_wait_limit_ns": (None, [C.c_uint64]),
        "h3fp4_status_string": (C.c_char_p, [i32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


# ------------------------------------------------------------------ marshalling helpers

def _ptr(t: Optional[torch.Tensor], what: str, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


_Tensor, _BF16, _F32, _I32, _U8 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _heads(t: torch.Tensor, what: str, rows: int, heads: int, d: int):
    """(address, row stride, head stride) of a bf16 [rows, heads, d] view: any row
    and head strides, the elements of a head contiguous."""
    try:
        row, head, one = t.stride()
        good = t.dtype is _BF16 and t.shape == (rows, heads, d) and t.is_cuda and (one == 1 or d == 1)
    except (AttributeError, ValueError):
        good = False
    if not good:
        _refuse_heads(t, what, rows, heads, d)
    # the stride of a dimension of one element says nothing about the memory
    if heads <= 1:
        head = d
    if rows <= 1:
        row = heads * head
    return t.data_ptr(), row, head


def _refuse_heads(t, what: str, rows: int, heads: int, d: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype is not _BF16:
        raise TypeError(f"{what} must be {_BF16}, got {t.dtype}")
    if t.shape != (rows, heads, d):
        raise ValueError(f"{what} must be {[rows, heads, d]}, got {list(t.shape)}")
    raise ValueError(f"{what}: the last dimension must be contiguous")


def _check_table(seq: Sequence[int]):
    if len(seq) < 2:
        raise ValueError(f"an offset table has two entries at least (0 first, the number of rows last), got {len(seq)}")


def _table(seq: Optional[Sequence[int]]):
    """(array of int64 to keep, its address, number of segments) of an offset table."""
    if seq is None:
        return None, None, 1
    _check_table(seq)
    a = array("q", seq if isinstance(seq, list) else [int(v) for v in seq])
    return a, a.buffer_info()[0], len(a) - 1


def _mask(t: Optional[torch.Tensor], what: str, n: int):
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype == torch.bool:
        t = t.view(torch.uint8)
    p = _ptr(t, what, torch.uint8)
    if t.numel() != n:
        raise ValueError(f"{what} must have {n} elements, got {t.numel()}")
    return p


def _f32(t: Optional[torch.Tensor], what: str, shape):
    if t is None:
        return None
    if isinstance(t, _Tensor) and t.dtype is _F32 and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, what, _F32)
    raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")


def _bf16(t: Optional[torch.Tensor], what: str, shape):
    if t is None:
        return None
    if isinstance(t, _Tensor) and t.dtype is _BF16 and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, what, _BF16)
    raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")


def _seg_pair(q_off, kv_off):
    if (q_off is None) != (kv_off is None):
        raise ValueError("q_off and kv_off go together")
    if q_off is not None and len(q_off) != len(kv_off):
        raise ValueError(f"q_off and kv_off must have the same length, got {len(q_off)} and {len(kv_off)}")
    keep_q, q, nseg = _table(q_off)
    keep_k, k, _ = _table(kv_off)
    return q, k, nseg, (keep_q, keep_k)


_raw_stream, _device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


def _stream(stream) -> Optional[int]:
    if stream is None:
        # the raw handle: torch.cuda.current_stream() builds a Stream object, 3 us per call
        return _raw_stream(_device()) if _raw_stream else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _segs(seg_off: Optional[Sequence[int]]):
    if seg_off is None:
        return None, 1, None
    _check_table(seg_off)
    arr = (C.c_int64 * len(seg_off))(*[int(v) for v in seg_off])
    return C.cast(arr, C.c_void_p), len(seg_off) - 1, arr


def _check(status: int, what: str):
    if status != 0:
        raise H3FP4Error(status, what)


def _workspace(ws: torch.Tensor, what: str = "ws") -> int:
    if isinstance(ws, _Tensor) and ws.dtype is _U8 and ws.is_cuda and ws.is_contiguous():
        return ws.data_ptr()
    return _ptr(ws, what, _U8)


# ------------------------------------------------------------------ C-ABI functions

def h3fp4_status_string(status: int) -> str:
    return load_library().h3fp4_status_string(status).decode()


def h3fp4_codes_bytes(rows: int, K: int) -> int:
    return int(load_library().h3fp4_codes_bytes(rows, K))


def h3fp4_sf_bytes(rows: int, K: int) -> int:
    return int(load_library().h3fp4_sf_bytes(rows, K))


def h3fp4_workspace_bytes(M: int, N: int, K: int, flags: int = 0) -> int:
    return int(load_library().h3fp4_workspace_bytes(M, N, K, flags))


def h3fp4_set_wait_limit_ns(ns: int) -> None:
    load_library().h3fp4_set_wait_limit_ns(int(ns))


def h3fp4_quantize_weight(w: torch.Tensor, codes: torch.Tensor, sf: torch.Tensor, gscale: torch.Tensor,
                          ws: torch.Tensor, stream=None) -> None:
    N, K = w.shape
    _check(load_library().h3fp4_quantize_weight(
        _ptr(w, "w", torch.bfloat16), N, K, _ptr(codes, "codes", torch.uint8), _ptr(sf, "sf", torch.uint8),
        _ptr(gscale, "gscale", torch.float32), _ptr(ws, "ws", torch.uint8), _stream(stream)),
        "h3fp4_quantize_weight")


def h3fp4_quantize_act(x: torch.Tensor, codes: torch.Tensor, sf: torch.Tensor, gscale: torch.Tensor,
                       ws: torch.Tensor, shift: Optional[torch.Tensor] = None,
                       scale: Optional[torch.Tensor] = None, seg_off: Optional[Sequence[int]] = None,
                       gscale_given: bool = False, stream=None) -> None:
    M, K = x.shape
    flags = (PROLOGUE_MOD if shift is not None else 0) | (GSCALE_GIVEN if gscale_given else 0)
    sp, nseg, _keep = _segs(seg_off)
    _check(load_library().h3fp4_quantize_act(
        _ptr(x, "x", torch.bfloat16), M, K, _ptr(shift, "shift", torch.float32),
        _ptr(scale, "scale", torch.float32), sp, nseg, _ptr(codes, "codes", torch.uint8),
        _ptr(sf, "sf", torch.uint8), _ptr(gscale, "gscale", torch.float32), flags,
        _ptr(ws, "ws", torch.uint8), _stream(stream)), "h3fp4_quantize_act")


def h3fp4_linear(x: torch.Tensor, w_codes: torch.Tensor, w_sf: torch.Tensor, w_gscale: torch.Tensor,
                 out: torch.Tensor, ws: torch.Tensor, *, K: Optional[int] = None,
                 a_sf: Optional[torch.Tensor] = None, a_gscale: Optional[torch.Tensor] = None,
                 shift: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                 gate: Optional[torch.Tensor] = None, resid: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, seg_off: Optional[Sequence[int]] = None,
                 gscale_given: bool = False, swiglu: bool = False, out_amax: bool = False,
                 fused: bool = False, stream=None) -> None:
    """out = [R + g*](alpha * NVFP4(prologue(x)) . W^T [+ b]).

    ``x`` is bf16 [M, K]; or uint8 codes [M, K/2] together with ``a_sf`` and
    ``a_gscale`` (pre-quantised activation).  ``swiglu``: out is [M, N/2] =
    bf16(silu(g) * u) over the weight's [gate 128 | up 128] row groups.
    ``out_amax``: also leave max|out| at :func:`h3fp4_ws_out_amax` (ws).
    ``fused``: the GEMM kernel quantises x itself (H3FP4_FUSED_QUANT).
    """
    prequant = x.dtype == torch.uint8
    M = x.shape[0]
    K = x.shape[1] * (2 if prequant else 1)
    N = out.shape[1] * (2 if swiglu else 1)
    flags = ((A_PREQUANT if prequant else 0) | (PROLOGUE_MOD if shift is not None else 0)
             | (EPI_BIAS if bias is not None else 0) | (EPI_GATE_RESID if gate is not None else 0)
             | (GSCALE_GIVEN if gscale_given else 0) | (EPI_SWIGLU if swiglu else 0)
             | (EPI_AMAX if out_amax else 0) | (FUSED_QUANT if fused else 0))
    sp, nseg, _keep = _segs(seg_off)
    _check(load_library().h3fp4_linear(
        _ptr(x, "x"), _ptr(a_sf, "a_sf", torch.uint8), _ptr(a_gscale, "a_gscale", torch.float32), M, N, K,
        _ptr(w_codes, "w_codes", torch.uint8), _ptr(w_sf, "w_sf", torch.uint8),
        _ptr(w_gscale, "w_gscale", torch.float32), _ptr(shift, "shift", torch.float32),
        _ptr(scale, "scale", torch.float32), _ptr(gate, "gate", torch.float32), sp, nseg,
        _ptr(bias, "bias", torch.bfloat16), _ptr(resid, "resid", torch.bfloat16),
        _ptr(out, "out", torch.bfloat16), flags, _ptr(ws, "ws", torch.uint8), _stream(stream)),
        "h3fp4_linear")


def h3fp4_linear_swiglu_nvfp4(x: torch.Tensor, w_codes: torch.Tensor, w_sf: torch.Tensor, w_gscale: torch.Tensor,
                              h_codes: torch.Tensor, h_sf: torch.Tensor, h_gscale: torch.Tensor, ws: torch.Tensor, *,
                              a_sf: Optional[torch.Tensor] = None, a_gscale: Optional[torch.Tensor] = None,
                              shift: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                              bias: Optional[torch.Tensor] = None, seg_off: Optional[Sequence[int]] = None,
                              gscale_given: bool = False, stream=None) -> None:
    """FC1 with the SwiGLU producer writing h = bf16(silu(g) * u) as NVFP4:
    ``h_codes`` uint8 [M, N/4], ``h_sf`` (h3fp4_sf_bytes(M, N/2)) under the
    given global scale ``h_gscale`` (device fp32 [1], an input)."""
    prequant = x.dtype == torch.uint8
    M = x.shape[0]
    K = x.shape[1] * (2 if prequant else 1)
    N = h_codes.shape[1] * 4
    flags = ((A_PREQUANT if prequant else 0) | (PROLOGUE_MOD if shift is not None else 0)
             | (EPI_BIAS if bias is not None else 0) | (GSCALE_GIVEN if gscale_given else 0))
    sp, nseg, _keep = _segs(seg_off)
    _check(load_library().h3fp4_linear_swiglu_nvfp4(
        _ptr(x, "x"), _ptr(a_sf, "a_sf", torch.uint8), _ptr(a_gscale, "a_gscale", torch.float32), M, N, K,
        _ptr(w_codes, "w_codes", torch.uint8), _ptr(w_sf, "w_sf", torch.uint8),
        _ptr(w_gscale, "w_gscale", torch.float32), _ptr(shift, "shift", torch.float32),
        _ptr(scale, "scale", torch.float32), sp, nseg, _ptr(bias, "bias", torch.bfloat16),
        _ptr(h_gscale, "h_gscale", torch.float32), _ptr(h_codes, "h_codes", torch.uint8),
        _ptr(h_sf, "h_sf", torch.uint8), flags, _ptr(ws, "ws", torch.uint8), _stream(stream)),
        "h3fp4_linear_swiglu_nvfp4")


def h3fp4_quantize_act_noalloc(x: torch.Tensor, codes: torch.Tensor, sf: torch.Tensor, gscale: torch.Tensor,
                               shift: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                               seg_off: Optional[Sequence[int]] = None, gscale_given: bool = False,
                               stream=None) -> None:
    """h3fp4_quantize_act without a workspace, for callers that may not allocate
    device memory; its scratch is a static device array shared by all calls
    (serialise calls that could overlap on the GPU)."""
    M, K = x.shape
    flags = (PROLOGUE_MOD if shift is not None else 0) | (GSCALE_GIVEN if gscale_given else 0)
    sp, nseg, _keep = _segs(seg_off)
    _check(load_library().h3fp4_quantize_act_noalloc(
        _ptr(x, "x", torch.bfloat16), M, K, _ptr(shift, "shift", torch.float32),
        _ptr(scale, "scale", torch.float32), sp, nseg, _ptr(codes, "codes", torch.uint8),
        _ptr(sf, "sf", torch.uint8), _ptr(gscale, "gscale", torch.float32), flags, _stream(stream)),
        "h3fp4_quantize_act_noalloc")


def h3fp4_act_amax(x: torch.Tensor, amax: torch.Tensor, ws: torch.Tensor, shift: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None, seg_off: Optional[Sequence[int]] = None,
                   stream=None) -> None:
    """amax of this call's (modulated) rows into ``amax`` (device fp32 [1])."""
    M, K = x.shape
    sp, nseg, _keep = _segs(seg_off)
    _check(load_library().h3fp4_act_amax(
        _ptr(x, "x", torch.bfloat16), M, K, _ptr(shift, "shift", torch.float32),
        _ptr(scale, "scale", torch.float32), sp, nseg, _ptr(amax, "amax", torch.float32),
        PROLOGUE_MOD if shift is not None else 0, _ptr(ws, "ws", torch.uint8), _stream(stream)),
        "h3fp4_act_amax")


def h3fp4_ws_out_amax(ws: torch.Tensor) -> torch.Tensor:
    """The fp32 [1] view of ``ws`` where an ``out_amax`` linear leaves max|out|."""
    addr = load_library().h3fp4_ws_out_amax(_ptr(ws, "ws", torch.uint8))
    off = int(addr) - ws.data_ptr()
    return ws[off:off + 4].view(torch.float32)


def h3fp4_gscale_from_amax(amax: torch.Tensor, gscale: torch.Tensor, stream=None) -> None:
    _check(load_library().h3fp4_gscale_from_amax(_ptr(amax, "amax", torch.float32),
                                                 _ptr(gscale, "gscale", torch.float32), _stream(stream)),
           "h3fp4_gscale_from_amax")


def h3fp4_selftest_timeout(ws: torch.Tensor, limit_ns: int, stream=None) -> None:
    _check(load_library().h3fp4_selftest_timeout(_ptr(ws, "ws", torch.uint8), int(limit_ns), _stream(stream)),
           "h3fp4_selftest_timeout")


def h3fp4_selftest_pack_timeout(x: torch.Tensor, a_gscale: torch.Tensor, ws: torch.Tensor, limit_ns: int,
                                stream=None) -> None:
    _check(load_library().h3fp4_selftest_pack_timeout(_ptr(x, "x", torch.bfloat16),
                                                      _ptr(a_gscale, "a_gscale", torch.float32),
                                                      _ptr(ws, "ws", torch.uint8), int(limit_ns), _stream(stream)),
           "h3fp4_selftest_pack_timeout")


def h3fp4_selftest_attn_timeout(ws: torch.Tensor, limit_ns: int, stream=None) -> None:
    if ws.numel() < 2048:
        raise ValueError("ws must have 2048 bytes")
    _check(load_library().h3fp4_selftest_attn_timeout(_ptr(ws, "ws", torch.uint8), int(limit_ns), _stream(stream)),
           "h3fp4_selftest_attn_timeout")


def h3fp4_measure_fp4_peak(ws: torch.Tensor, iters: int = 20000) -> float:
    """Measured FP4 MMA ceiling (TFLOP/s) of the current device (synchronous)."""
    out = C.c_float(0.0)
    _check(load_library().h3fp4_measure_fp4_peak(int(iters), C.byref(out), _ptr(ws, "ws", torch.uint8)),
           "h3fp4_measure_fp4_peak")
    return float(out.value)


def h3fp4_measure_fp4_pair_peak(ws: torch.Tensor, iters: int = 20000) -> float:
    """Measured ceiling (TFLOP/s) of the paired (2-CTA) FP4 MMA the GEMM issues (synchronous)."""
    out = C.c_float(0.0)
    _check(load_library().h3fp4_measure_fp4_pair_peak(int(iters), C.byref(out), _ptr(ws, "ws", torch.uint8)),
           "h3fp4_measure_fp4_pair_peak")
    return float(out.value)


MMA_FORMS = {0: "cta_group::1 M=128 N=256 K=64, A smem", 1: "cta_group::2 M=256 N=256 K=64, A smem",
             2: "cta_group::1, A TMEM", 3: "cta_group::2, A TMEM", 4: "cta_group::1, 2 x N=128 sharing A",
             5: "cta_group::1, 2 x N=128, collector::a fill/lastuse", 6: "cta_group::2, 2 x N=128 sharing A"}


def h3fp4_measure_fp4_form(ws: torch.Tensor, form: int, iters: int = 20000) -> float:
    """Measured ceiling (TFLOP/s) of one kind::mxf4nvf4 MMA form (MMA_FORMS; synchronous)."""
    out = C.c_float(0.0)
    _check(load_library().h3fp4_measure_fp4_form(int(form), int(iters), C.byref(out), _ptr(ws, "ws", torch.uint8)),
           "h3fp4_measure_fp4_form")
    return float(out.value)


def h3fp4_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_out: torch.Tensor,
                       k_out: Optional[torch.Tensor], *, q_weight: Optional[torch.Tensor] = None,
                       k_weight: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                       sin: Optional[torch.Tensor] = None, interleaved: bool = False,
                       seg_off: Optional[Sequence[int]] = None, eps: float = 1e-6, stream=None) -> None:
    """Per-head RMS norm and rotation of Q [M, Hq, D] and K [M, Hk, D] (bf16, row
    and head strides positive multiples of 8; ``k`` and ``k_out`` may be None) in
    one pass.

    ``q_weight`` / ``k_weight``: fp32 [nseg, D]; ``cos`` / ``sin``: fp32
    [M, rot/2].  The rotated pairs are (i, i + rot/2), or (2i, 2i + 1) with
    ``interleaved``.  An output may be its own input."""
    M, Hq, D = q.shape
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    Hk = k.shape[1] if k is not None else 0
    keep, sp, nseg = _table(seg_off)
    half = cos.shape[-1] if cos is not None else 0
    views = [*_heads(q, "q", M, Hq, D), *_heads(q_out, "q_out", M, Hq, D)]
    if k is not None:
        views += (*_heads(k, "k", M, Hk, D), *_heads(k_out, "k_out", M, Hk, D))
    a = array("q", views)   # h3fp4_heads, one after the other
    at = a.buffer_info()[0]
    _check(load_library().h3fp4_qk_norm_rope(
        at, at + 48 if k is not None else None, M, Hq, Hk, D, _f32(q_weight, "q_weight", (nseg, D)),
        _f32(k_weight, "k_weight", (nseg, D)), _f32(cos, "cos", (M, half)), _f32(sin, "sin", (M, half)), 2 * half,
        sp, nseg, eps, at + 24, at + 72 if k is not None else None, ROPE_PAIRS if interleaved else 0,
        _stream(stream)), "h3fp4_qk_norm_rope")


def h3fp4_cross_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, *,
                     q_off: Optional[Sequence[int]] = None, kv_off: Optional[Sequence[int]] = None,
                     key_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """out [M, Hq, D] = attention of q [M, Hq, D] to k, v [T, Hkv, D] (bf16; row and
    head strides are positive multiples of 8, so shared key heads are given once
    and not expanded), segment by segment of ``q_off`` / ``kv_off``.

    ``key_mask``: bool or uint8 [T], False / 0 leaves a key out; ``scale``
    defaults to 1/sqrt(D); ``lse``: fp32 [M, Hq], also written.  ``ws`` from
    :func:`alloc_attn_workspace`."""
    M, Hq, D = q.shape
    T, Hkv, _ = k.shape
    qp, kp, nseg, keep = _seg_pair(q_off, kv_off)
    a = array("q", (*_heads(q, "q", M, Hq, D), *_heads(k, "k", T, Hkv, D), *_heads(v, "v", T, Hkv, D),
                    *_heads(out, "out", M, Hq, D)))
    at = a.buffer_info()[0]
    _check(load_library().h3fp4_cross_attn(
        at, at + 24, at + 48, M, T, Hq, Hkv, D, qp, kp, nseg, _mask(key_mask, "key_mask", T),
        D ** -0.5 if scale is None else scale, at + 72, _f32(lse, "lse", (M, Hq)), _workspace(ws), ws.numel(),
        _stream(stream)), "h3fp4_cross_attn")


def h3fp4_shared_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_ctx: torch.Tensor, v_ctx: torch.Tensor,
                      out: torch.Tensor, ws: torch.Tensor, *, q_off: Optional[Sequence[int]] = None,
                      kv_off: Optional[Sequence[int]] = None, key_mask: Optional[torch.Tensor] = None,
                      ctx_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                      lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """:func:`h3fp4_cross_attn` with a context ``k_ctx``, ``v_ctx`` [C, Hkv, D]
    that the rows of every segment attend to beside their own keys, in one
    softmax; ``ctx_mask``: bool or uint8 [C]."""
    M, Hq, D = q.shape
    T, Hkv, _ = k.shape
    ctx = k_ctx.shape[0]
    qp, kp, nseg, keep = _seg_pair(q_off, kv_off)
    a = array("q", (*_heads(q, "q", M, Hq, D), *_heads(k, "k", T, Hkv, D), *_heads(v, "v", T, Hkv, D),
                    *_heads(k_ctx, "k_ctx", ctx, Hkv, D), *_heads(v_ctx, "v_ctx", ctx, Hkv, D),
                    *_heads(out, "out", M, Hq, D)))
    at = a.buffer_info()[0]
    _check(load_library().h3fp4_shared_attn(
        at, at + 24, at + 48, at + 72, at + 96, M, T, ctx, Hq, Hkv, D, qp, kp, nseg, _mask(key_mask, "key_mask", T),
        _mask(ctx_mask, "ctx_mask", ctx), D ** -0.5 if scale is None else scale, at + 120,
        _f32(lse, "lse", (M, Hq)), _workspace(ws), ws.numel(), _stream(stream)), "h3fp4_shared_attn")


def h3fp4_attn_workspace_bytes(M: int, T: int, Hq: int, Hkv: int, D: int, q_off: Optional[Sequence[int]] = None,
                               kv_off: Optional[Sequence[int]] = None, ctx: int = 0) -> int:
    qp, kp, nseg, _keep = _seg_pair(q_off, kv_off)
    return int(load_library().h3fp4_attn_workspace_bytes(M, T, ctx, Hq, Hkv, D, qp, kp, nseg))


def h3fp4_block_norm(x: torch.Tensor, out: Optional[torch.Tensor] = None, *, y: Optional[torch.Tensor] = None,
                     x_out: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                     y_weight: Optional[torch.Tensor] = None, x_scale: float = 1.0,
                     weight: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                     scale: Optional[torch.Tensor] = None, seg_off: Optional[Sequence[int]] = None,
                     eps: float = 1e-6, post_norm: bool = False, layer_norm: bool = False,
                     out_amax: Optional[torch.Tensor] = None, stream=None) -> None:
    """The norms around a block with its gate and residual, one pass over the rows of bf16 [M, K]:

    ``r = x_scale * x + gate * y'`` into ``x_out``, with ``y' = y`` or (``post_norm``) its RMS norm times
    ``y_weight``; the RMS norm of r (``layer_norm``: its layer norm) times ``weight``, modulated by ``1 + scale`` and
    ``shift``, into ``out``.  The vectors are fp32 [nseg, K], each may be None; without ``y`` r is x.  ``out_amax``:
    fp32 [1], receives max|out|.  An output may be its own input."""
    M, K = shape = x.shape
    keep, sp, nseg = _table(seg_off)
    vec = (nseg, K)
    _check(load_library().h3fp4_block_norm(
        _bf16(x, "x", shape), _bf16(y, "y", shape), M, K, _f32(y_weight, "y_weight", vec), _f32(gate, "gate", vec),
        x_scale, _f32(weight, "weight", vec), _f32(shift, "shift", vec), _f32(scale, "scale", vec), sp, nseg, eps,
        _bf16(x_out, "x_out", shape), _bf16(out, "out", shape), _f32(out_amax, "out_amax", (1,)),
        (NORM_POST if post_norm else 0) | (NORM_LAYER if layer_norm else 0), _stream(stream)), "h3fp4_block_norm")


def h3fp4_linear_rows(x: torch.Tensor, w_codes: torch.Tensor, w_sf: torch.Tensor, w_gscale: torch.Tensor,
                      out: torch.Tensor, ws: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, resid: Optional[torch.Tensor] = None, swiglu: bool = False,
                      stream=None) -> None:
    """out = [resid + gate *](x . W^T [+ bias]) of a few rows x bf16 [M, K] (M <= ROWS_MAX) over NVFP4 weights; x is not
    quantised.

    ``gate``: fp32 [M, N], or [N] for all rows, with ``resid`` bf16 [M, N] (which may be ``out``).  ``swiglu``: out is
    [M, N/2] = bf16(silu(g) * u) over the weight's [gate 128 | up 128] row groups.  ``ws`` from
    :func:`alloc_rows_workspace`."""
    M, K = x.shape
    N = out.shape[1] * (2 if swiglu else 1)
    stride = 0
    if gate is not None:
        stride = N if gate.dim() == 2 else 0
        gate_shape = (M, N) if stride else (N,)
    if w_codes.shape != (N, K // 2):
        raise ValueError(f"w_codes must be {[N, K // 2]}, got {list(w_codes.shape)}")
    if w_sf.numel() != (N + 127) // 128 * 8 * K:
        raise ValueError(f"w_sf must have {(N + 127) // 128 * 8 * K} elements, got {w_sf.numel()}")
    flags = ((EPI_BIAS if bias is not None else 0) | (EPI_GATE_RESID if gate is not None else 0)
             | (EPI_SWIGLU if swiglu else 0))
    _check(load_library().h3fp4_linear_rows(
        _bf16(x, "x", x.shape), M, N, K, _ptr(w_codes, "w_codes", torch.uint8), _ptr(w_sf, "w_sf", torch.uint8),
        _f32(w_gscale, "w_gscale", (1,)), None if gate is None else _f32(gate, "gate", gate_shape), stride,
        _bf16(bias, "bias", (N,)), _bf16(resid, "resid", (M, N)), _bf16(out, "out", (M, N // 2 if swiglu else N)), flags,
        _workspace(ws), ws.numel(), _stream(stream)), "h3fp4_linear_rows")


def h3fp4_selftest_linear_rows_timeout(ws: torch.Tensor, limit_ns: int, stream=None) -> None:
    if ws.numel() < h3fp4_linear_rows_workspace_bytes(64, 128, 1024):
        raise ValueError("ws must be a workspace for 64 rows of 1024 columns and 128 outputs")
    _check(load_library().h3fp4_selftest_linear_rows_timeout(_ptr(ws, "ws", torch.uint8), int(limit_ns),
                                                             _stream(stream)), "h3fp4_selftest_linear_rows_timeout")


def h3fp4_linear_rows_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load_library().h3fp4_linear_rows_workspace_bytes(M, N, K))


def _i32(t: Optional[torch.Tensor], what: str, shape):
    if t is None:
        return 0
    if isinstance(t, _Tensor) and t.dtype is _I32 and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, what, _I32)
    raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")


def _cache_width(D: int) -> int:
    return 64 if D <= 64 else 128 if D <= 128 else 256


def _cache(cache: torch.Tensor, table: torch.Tensor, length: torch.Tensor, row_off: Optional[torch.Tensor], M: int,
           D: int, k_gscale: Optional[torch.Tensor], v_gscale: Optional[torch.Tensor]):
    """The fields of an h3fp4_cache, and its number of heads."""
    at = _workspace(cache, "cache")
    width = 72 if D <= 64 else 144 if D <= 128 else 288                # nine eighths of the room of a head
    try:
        n_pages, heads, page, held = cache.shape
    except ValueError:
        held = None
    if held != width:
        raise ValueError(f"cache must be [pages, heads, page, {width}] for heads of {D}, got {list(cache.shape)}")
    try:
        nseq, max_pages = shape = table.shape
    except (AttributeError, ValueError):
        raise ValueError("table must be an int32 tensor [nseq, max_pages]") from None
    if row_off is None and nseq != M:
        raise ValueError(f"without row_off there is one row per sequence: {M} rows, {nseq} sequences")
    of_heads = (heads,)
    return (at, n_pages, page, heads, D, _i32(table, "table", shape), max_pages, _i32(length, "length", (nseq,)),
            _i32(row_off, "row_off", (nseq + 1,)), nseq, _f32(k_gscale, "k_gscale", of_heads) or 0,
            _f32(v_gscale, "v_gscale", of_heads) or 0), heads


def _cache_rows(name: str, k, v, cache, table, length, row_off, k_gscale, v_gscale, stream):
    M, heads, D = k.shape
    fields, held = _cache(cache, table, length, row_off, M, D, k_gscale, v_gscale)
    if heads != held:
        raise ValueError(f"cache holds {held} heads, the rows have {heads}")
    a = array("q", (*_heads(k, "k", M, heads, D), *_heads(v, "v", M, heads, D), *fields))
    at = a.buffer_info()[0]
    _check(getattr(load_library(), name)(at, at + 24, M, at + 48, _stream(stream)), name)


def h3fp4_cache_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, table: torch.Tensor,
                       length: torch.Tensor, row_off: Optional[torch.Tensor] = None, *,
                       k_gscale: Optional[torch.Tensor] = None, v_gscale: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """Write the rows ``k``, ``v`` [M, heads, D] (bf16 views) to their places in a paged 4-bit ``cache`` of
    :func:`alloc_kv_cache`.

    ``table`` int32 [nseq, max_pages]: the pages of each sequence; ``length`` int32 [nseq]: its tokens, with the new
    ones; ``row_off`` int32 [nseq + 1]: which rows are its last ones (None: row s is sequence s's).  All on the device,
    read when the call runs.  ``k_gscale`` / ``v_gscale``: fp32 [heads]."""
    _cache_rows("h3fp4_cache_append", k, v, cache, table, length, row_off, k_gscale, v_gscale, stream)


def h3fp4_cache_read(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, length: torch.Tensor,
                     row_off: Optional[torch.Tensor] = None, *, k_gscale: Optional[torch.Tensor] = None,
                     v_gscale: Optional[torch.Tensor] = None, stream=None) -> None:
    """The way back of :func:`h3fp4_cache_append`: the rows' places as bf16 into ``k``, ``v``."""
    _cache_rows("h3fp4_cache_read", k, v, cache, table, length, row_off, k_gscale, v_gscale, stream)


def h3fp4_cache_attn(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, length: torch.Tensor, out: torch.Tensor,
                     ws: torch.Tensor, *, row_off: Optional[torch.Tensor] = None,
                     k_gscale: Optional[torch.Tensor] = None, v_gscale: Optional[torch.Tensor] = None,
                     causal: bool = True, scale: Optional[float] = None, lse: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """out [M, Hq, D] = attention of the rows q [M, Hq, D] to the cached keys and values of their sequences
    (arguments as in :func:`h3fp4_cache_append`), up to each row's own position with ``causal``, else to all.

    ``scale`` defaults to 1/sqrt(D); ``lse``: fp32 [M, Hq], also written.  ``ws`` from
    :func:`alloc_cache_attn_workspace`."""
    M, Hq, D = q.shape
    fields, _ = _cache(cache, table, length, row_off, M, D, k_gscale, v_gscale)
    a = array("q", (*_heads(q, "q", M, Hq, D), *_heads(out, "out", M, Hq, D), *fields))
    at = a.buffer_info()[0]
    _check(load_library().h3fp4_cache_attn(
        at, M, Hq, at + 48, D ** -0.5 if scale is None else scale, at + 24, _f32(lse, "lse", (M, Hq)),
        CAUSAL if causal else 0, _workspace(ws), ws.numel(), _stream(stream)), "h3fp4_cache_attn")


def h3fp4_cache_page_bytes(heads: int, D: int, page: int) -> int:
    return int(load_library().h3fp4_cache_page_bytes(heads, D, page))


def h3fp4_cache_attn_workspace_bytes(D: int) -> int:
    return int(load_library().h3fp4_cache_attn_workspace_bytes(D))


def h3fp4_selftest_cache_attn_timeout(ws: torch.Tensor, limit_ns: int, stream=None) -> None:
    if ws.numel() < h3fp4_cache_attn_workspace_bytes(64):
        raise ValueError("ws must be a workspace for heads of 64")
    _check(load_library().h3fp4_selftest_cache_attn_timeout(_ptr(ws, "ws", torch.uint8), int(limit_ns),
                                                            _stream(stream)), "h3fp4_selftest_cache_attn_timeout")


def h3fp4_check(ws: torch.Tensor, stream=None) -> None:
    """Synchronise and raise H3FP4Error if a device wait timed out."""
    _check(load_library().h3fp4_check(_ptr(ws, "ws", torch.uint8), _stream(stream)), "h3fp4_check")


# ------------------------------------------------------------------ buffer helpers (torch allocations)

def alloc_nvfp4(rows: int, K: int, device="cuda"):
    """(codes uint8 [rows, K/2], sf uint8 [sf_bytes], gscale fp32 [1]) on ``device``."""
    return (torch.empty((rows, K // 2), dtype=torch.uint8, device=device),
            torch.empty(h3fp4_sf_bytes(rows, K), dtype=torch.uint8, device=device),
            torch.empty(1, dtype=torch.float32, device=device))


def alloc_workspace(M: int, N: int, K: int, flags: int = 0, device="cuda") -> torch.Tensor:
    return torch.zeros(h3fp4_workspace_bytes(M, N, K, flags), dtype=torch.uint8, device=device)


def alloc_attn_workspace(M: int, T: int, Hq: int, Hkv: int, D: int, q_off: Optional[Sequence[int]] = None,
                         kv_off: Optional[Sequence[int]] = None, ctx: int = 0, device="cuda") -> torch.Tensor:
    """Workspace of the attention calls for these sizes (``ctx``: rows of the shared context)."""
    n = h3fp4_attn_workspace_bytes(M, T, Hq, Hkv, D, q_off, kv_off, ctx)
    if n == 0:
        raise ValueError("sizes or segment tables that the attention calls refuse")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_rows_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """Workspace of :func:`h3fp4_linear_rows` for these sizes."""
    n = h3fp4_linear_rows_workspace_bytes(M, N, K)
    if n == 0:
        raise ValueError("sizes that the linear of a few rows refuses")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_kv_cache(pages: int, heads: int, D: int, page: int = 64, device="cuda") -> torch.Tensor:
    """uint8 [pages, heads, page, bytes of a token and head]: a paged 4-bit cache of ``pages`` pages of ``page`` tokens."""
    if h3fp4_cache_page_bytes(heads, D, page) == 0:
        raise ValueError("sizes that the cache calls refuse")
    return torch.zeros(pages, heads, page, _cache_width(D) * 9 // 8, dtype=torch.uint8, device=device)


def alloc_cache_attn_workspace(rows: int, seqs: int, Hq: int, heads: int, D: int, device="cuda") -> torch.Tensor:
    """Workspace of :func:`h3fp4_cache_attn` (its size depends on D alone)."""
    n = h3fp4_cache_attn_workspace_bytes(D)
    if n == 0 or heads < 1 or Hq % heads or seqs < 1 or rows < 0:
        raise ValueError("sizes that the cache attention refuses")
    return torch.zeros(n, dtype=torch.uint8, device=device)
