"""Python binding of libqlin.so (quantized decoder projections on MI355X).

Argument marshalling only: every function below forwards device pointers,
sizes and the current HIP stream to the C ABI declared in include/qlin.h and
raises QlinError on a non-OK status.  torch supplies memory and streams; no
computation happens here.  If the library is not built, importing this package
fails loudly -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlin.so")

(QLIN_OK, QLIN_ERR_NULL, QLIN_ERR_SHAPE, QLIN_ERR_ALIGN, QLIN_ERR_UNSUPPORTED, QLIN_ERR_HIP, QLIN_ERR_ALIAS,
 QLIN_ERR_TOO_LARGE) = range(8)
OUT_BF16, OUT_I32, OUT_F32 = 0, 1, 2
SCHEME_W8A8, SCHEME_FP8_ROWWISE, SCHEME_FP8_BLOCK = 0, 1, 2
MAX_SEGMENTS = 4
PATH_AUTO, PATH_GEMV, PATH_SMALL, PATH_LARGE = 0, 1, 2, 3
# the tiled GEMM with a fixed output tile (weight rows x tokens)
PATH_LARGE_256X128, PATH_LARGE_128X128, PATH_LARGE_128X64, PATH_LARGE_128X256 = 4, 5, 6, 7
PATH_LARGE_128X128_K2, PATH_LARGE_128X64_K2 = 8, 9
PATH_LARGE_256X256_W8 = 10   # int8 and FP8 rowwise only
PATH_LARGE_256X256 = 11      # int8 and FP8 rowwise only
ABI_VERSION = 5
NOALLOC_MAX_CODE_BYTES = 16 << 20    # staging capacity of qlin_linear_noalloc
NOALLOC_MAX_SCALES = 1 << 20
MAX_K = 131072

# Exported symbols and their C signatures (restype, argtypes).
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_S = ctypes.c_int
SIGNATURES = {
    "qlin_quant_act_int8": (_S, [_P, _I64, _I64, _P, _P, _P]),
    "qlin_quant_act_fp8": (_S, [_P, _I64, _I64, _I32, _P, _P, _P]),
    "qlin_gemv_w8a8": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _S, _P]),
    "qlin_gemm_w8a8": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _P]),
    "qlin_gemm_w8a8_ex": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _S, _P]),
    "qlin_gemm_fp8_rowwise": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _P]),
    "qlin_gemm_fp8_rowwise_ex": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _S, _P]),
    "qlin_gemm_fp8_block": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _P]),
    "qlin_gemm_fp8_block_ex": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _S, _P]),
    "qlin_linear": (_S, [_S, _P, _I64, _I64, _P, _I32, _S, _P, _P, _P]),
    "qlin_linear_weight_only": (_S, [_S, _P, _I64, _I64, _P, _I32, _S, _P]),
    "qlin_linear_swiglu": (_S, [_S, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _P, _P]),
    "qlin_linear_noalloc": (_S, [_S, _P, _I64, _I64, _P, _I32, _S, _P]),
    "qlin_pack_weights": (_S, [_S, _P, _I64, _I64, _P, _P]),
    "qlin_linear_packed": (_S, [_S, _P, _I64, _I64, _P, _I32, _S, _P, _P, _P]),
    "qlin_linear_swiglu_packed": (_S, [_S, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _P, _P]),
    "qlin_status_string": (ctypes.c_char_p, [_S]),
    "qlin_abi_version": (_S, []),
    "qlin_last_hip_error": (_S, []),
}

# include/qlin_w4.h: 4-bit weights, routing, experts
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
MAX_EXPERTS, MAX_CHOICES, MAX_GROUPS = 1024, 32, 64
_F = ctypes.c_float
SIGNATURES_W4 = {
    "qlin_w4_packed_bytes": (_I64, [_I64, _I64]),
    "qlin_w4_packed_scales": (_I64, [_I64, _I64, _I32]),
    "qlin_pack_w4": (_S, [_P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P, _P]),
    "qlin_linear_w4": (_S, [_P, _I64, _I64, _I32, _P, _P, _I32, _S, _P]),
    "qlin_linear_swiglu_w4": (_S, [_P, _I64, _I64, _I32, _P, _P, _P, _P]),
    "qlin_route": (_S, [_P, _S, _I64, _I64, _I32, _S, _P, _I32, _I32, _I32, _I32, _F, _P, _P, _P]),
    "qlin_experts_w4_workspace": (_I64, [_I64, _I32, _I64, _I64, _I64]),
    "qlin_experts_w4": (_S, [_P, _I64, _I64, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P]),
}

# include/qlin_layer.h: norm, rotary positions, cache, attention of one token
CACHE_BF16, CACHE_INT8, CACHE_FP8 = 0, 1, 2
MAX_HEADS, MAX_HEAD_DIM = 1024, 256
SIGNATURES_LAYER = {
    "qlin_norm_bf16": (_S, [_P, _P, _P, _I64, _I64, _F, _P, _P, _P]),
    "qlin_norm_int8": (_S, [_P, _P, _P, _I64, _I64, _F, _P, _P, _P, _P]),
    "qlin_norm_fp8": (_S, [_P, _P, _P, _I64, _I64, _F, _I32, _P, _P, _P, _P]),
    "qlin_rope": (_S, [_P, _I64, _P, _I64, _I32, _I32, _P, _P, _F, _P, _I64, _P]),
    "qlin_cache_write": (_S, [_P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _F, _P, _P]),
    "qlin_cache_read": (_S, [_P, _P, _I64, _P, _P, _P]),
    "qlin_attn_decode_workspace": (_I64, [_I32, _I32, _I32]),
    "qlin_attn_decode": (_S, [_P, _P, _P, _I64, _I32, _I64, _P, _I64, _F, _P, _P, _P]),
}


class QlinRotation(ctypes.Structure):
    """struct qlin_rotation."""
    _fields_ = [("frequencies", ctypes.c_void_p), ("dims", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("strength", ctypes.c_float)]


class QlinKVCache(ctypes.Structure):
    """struct qlin_kv_cache: the keys and values of one layer."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("kind", ctypes.c_int32)]


class QlinQueries(ctypes.Structure):
    """struct qlin_queries: the queries of a qlin_cache_write."""
    _fields_ = [("q", ctypes.c_void_p), ("stride", ctypes.c_int64), ("gamma", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


class QlinW4Weight(ctypes.Structure):
    """struct qlin_w4_weight: one packed 4-bit matrix, or one per expert."""
    _fields_ = [("q_w", ctypes.c_void_p), ("s_w", ctypes.c_void_p), ("z_w", ctypes.c_void_p), ("n", ctypes.c_int64)]


class QlinSegment(ctypes.Structure):
    """struct qlin_segment: one weight matrix reading the call's activations."""
    _fields_ = [("q_w", ctypes.c_void_p), ("s_w", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n", ctypes.c_int64)]


class QlinError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.qlin_status_string(status).decode() if _lib is not None else str(status)
        if status == QLIN_ERR_HIP:
            msg += f" (hip error {_lib.qlin_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def _load():
    # torch is imported first so that libqlin.so binds (by soname) to the HIP
    # runtime torch already loaded: one runtime per process, shared streams.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python quantized_linear_layers_token_amd/build.py` "
            "(the HIP library is the only implementation; there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    if lib.qlin_abi_version() != ABI_VERSION:      # (int and no arguments: ctypes' default) before a symbol can be missing
        raise ImportError(f"libqlin ABI {lib.qlin_abi_version()} != binding ABI {ABI_VERSION}")
    for name, (res, args) in {**SIGNATURES, **SIGNATURES_W4, **SIGNATURES_LAYER}.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def lib():
    """The raw ctypes handle of libqlin.so."""
    return _lib


def _check(status: int, where: str):
    if status != QLIN_OK:
        raise QlinError(status, where)


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dims2(t, name, elem=None):
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor")
    if elem is not None and t.element_size() != elem:
        raise ValueError(f"{name} must have {elem}-byte elements, not {t.element_size()}")
    return t.shape[0], t.shape[1]


def _out_bytes(out):
    return 2 if out == OUT_BF16 else 4


def _args(*items):
    """Checks every tensor argument before its address reaches the library,
    which sees only pointers: (name, tensor, bytes the call reads or writes,
    required element size or None).  A tensor must be contiguous and hold at
    least that many bytes, and all of them must be device tensors.  Optional
    arguments (None) are left to the library, which returns QLIN_ERR_NULL
    where one is required."""
    given = [(n, t, b, e) for n, t, b, e in items if t is not None]
    for name, t, nbytes, elem in given:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if elem is not None and t.element_size() != elem:
            raise ValueError(f"{name} must have {elem}-byte elements, not {t.element_size()}")
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise ValueError(f"{name} holds {have} bytes; the call accesses {nbytes}")
    for name, t, _, _ in given:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")


def _sx_count(scheme_block, M, K):
    return M * (K // 128) if scheme_block else M


def _sw_count(scheme_block, N, K):
    return (N // 128) * (K // 128) if scheme_block else N


# --------------------------------------------------------------------------
# Quantizers
# --------------------------------------------------------------------------

def qlin_quant_act_int8(x, q, s, stream=None):
    """x: bf16 (or int16 bit patterns) [M, K]; q: int8 [M, K]; s: f32 [M]."""
    M, K = _dims2(x, "x", 2)
    _args(("q", q, M * K, 1), ("s", s, 4 * M, 4), ("x", x, 0, None))
    _check(_lib.qlin_quant_act_int8(_ptr(x), M, K, _ptr(q), _ptr(s), _stream(stream)), "qlin_quant_act_int8")


def qlin_quant_act_fp8(x, q, s, group=0, stream=None):
    """x: bf16 [M, K]; q: uint8 E4M3 codes [M, K]; s: f32 [M] (group 0) or [M, K/128] (group 128)."""
    M, K = _dims2(x, "x", 2)
    _args(("q", q, M * K, 1), ("s", s, 4 * _sx_count(group == 128, M, K), 4), ("x", x, 0, None))
    _check(_lib.qlin_quant_act_fp8(_ptr(x), M, K, group, _ptr(q), _ptr(s), _stream(stream)), "qlin_quant_act_fp8")


# --------------------------------------------------------------------------
# Products
# --------------------------------------------------------------------------

def qlin_gemv_w8a8(q_x, s_x, q_w, s_w, y, out=OUT_BF16, stream=None):
    """q_x int8 [K] or [1, K]; s_x f32 [1]; q_w int8 [N, K]; s_w bf16 [N]; y [N] or [1, N]."""
    N, K = _dims2(q_w, "q_w", 1)
    _args(("q_x", q_x, K, 1), ("s_x", s_x, 4, 4), ("s_w", s_w, 2 * N, 2), ("y", y, N * _out_bytes(out), None),
          ("q_w", q_w, 0, None))
    _check(_lib.qlin_gemv_w8a8(_ptr(q_x), _ptr(s_x), _ptr(q_w), _ptr(s_w), _ptr(y), N, K, out, _stream(stream)),
           "qlin_gemv_w8a8")


def _mnk(q_x, q_w, s_x, s_w, y, out, block=False):
    M, K = _dims2(q_x, "q_x", 1)
    N, K2 = _dims2(q_w, "q_w", 1)
    if K != K2:
        raise ValueError(f"K mismatch: q_x has {K}, q_w has {K2}")
    _args(("s_x", s_x, 4 * _sx_count(block, M, K), 4), ("s_w", s_w, 2 * _sw_count(block, N, K), 2),
          ("y", y, M * N * _out_bytes(out), None), ("q_x", q_x, 0, None), ("q_w", q_w, 0, None))
    return M, N, K


def qlin_gemm_w8a8(q_x, s_x, q_w, s_w, y, out=OUT_BF16, path=PATH_AUTO, stream=None):
    """q_x int8 [M, K]; s_x f32 [M]; q_w int8 [N, K]; s_w bf16 [N]; y [M, N] (bf16 / i32 / f32)."""
    M, N, K = _mnk(q_x, q_w, s_x, s_w, y, out)
    _check(_lib.qlin_gemm_w8a8_ex(_ptr(q_x), _ptr(s_x), _ptr(q_w), _ptr(s_w), _ptr(y), M, N, K, out, path,
                                  _stream(stream)), "qlin_gemm_w8a8")


def qlin_gemm_fp8_rowwise(q_x, s_x, q_w, s_w, y, out=OUT_BF16, path=PATH_AUTO, stream=None):
    """q_x uint8 E4M3 [M, K]; s_x f32 [M]; q_w uint8 E4M3 [N, K]; s_w bf16 [N]; y [M, N]."""
    M, N, K = _mnk(q_x, q_w, s_x, s_w, y, out)
    _check(_lib.qlin_gemm_fp8_rowwise_ex(_ptr(q_x), _ptr(s_x), _ptr(q_w), _ptr(s_w), _ptr(y), M, N, K, out, path,
                                         _stream(stream)), "qlin_gemm_fp8_rowwise")


def qlin_gemm_fp8_block(q_x, s_x, q_w, s_w, y, out=OUT_BF16, path=PATH_AUTO, stream=None):
    """q_x uint8 E4M3 [M, K]; s_x f32 [M, K/128]; q_w uint8 E4M3 [N, K]; s_w bf16 [N/128, K/128]; y [M, N]."""
    M, N, K = _mnk(q_x, q_w, s_x, s_w, y, out, block=True)
    _check(_lib.qlin_gemm_fp8_block_ex(_ptr(q_x), _ptr(s_x), _ptr(q_w), _ptr(s_w), _ptr(y), M, N, K, out, path,
                                       _stream(stream)), "qlin_gemm_fp8_block")


def status_string(status: int) -> str:
    return _lib.qlin_status_string(status).decode()


# --------------------------------------------------------------------------
# Fused projection (bf16 activations in)
# --------------------------------------------------------------------------

def _segment_args(scheme, M, K, segments, out):
    """The _args items of the segments' tensors (shapes checked here)."""
    block = scheme == SCHEME_FP8_BLOCK
    items = []
    for i, (qw, sw, y) in enumerate(segments):
        n, k2 = _dims2(qw, f"segment {i} q_w", 1)
        if k2 != K:
            raise ValueError("every q_w must be [n, K]")
        items += [(f"segment {i} s_w", sw, 2 * _sw_count(block, n, K), 2),
                  (f"segment {i} y", y, M * n * _out_bytes(out), None), (f"segment {i} q_w", qw, 0, None)]
    return items


def segments_array(segments):
    """[(q_w [n, K], s_w, y), ...] -> ctypes array of QlinSegment."""
    arr = (QlinSegment * len(segments))()
    for i, (qw, sw, y) in enumerate(segments):
        arr[i] = QlinSegment(_ptr(qw), _ptr(sw), _ptr(y), qw.shape[0])
    return arr


def qlin_linear(scheme, x, segments, out=OUT_BF16, q_x=None, s_x=None, stream=None):
    """x bf16 [M, K]; segments: list of (q_w [n, K], s_w, y [M, n]) sharing x.
    q_x / s_x: staging for the quantized activations (optional where one launch
    does the whole call: M == 1, the two-token form, or M <= 4 with K <= 4096)."""
    M, K = _dims2(x, "x", 2)
    block = scheme == SCHEME_FP8_BLOCK
    _args(*_segment_args(scheme, M, K, segments, out), ("q_x", q_x, M * K, 1),
          ("s_x", s_x, 4 * _sx_count(block, M, K), 4), ("x", x, 0, None))
    arr = segments_array(segments)
    _check(_lib.qlin_linear(scheme, _ptr(x), M, K, arr, len(segments), out, _ptr(q_x), _ptr(s_x),
                            _stream(stream)), "qlin_linear")


def qlin_pack_weights(scheme, q_w, q_w_packed, stream=None):
    """Reorders q_w [N, K] (1-byte codes, row-major) into the matrix-core
    operand order of qlin_linear_packed, written to q_w_packed (N * K bytes,
    e.g. a tensor like q_w).  Any scheme; N and K multiples of 128."""
    N, K = _dims2(q_w, "q_w", 1)
    _args(("q_w_packed", q_w_packed, N * K, 1), ("q_w", q_w, 0, None))
    _check(_lib.qlin_pack_weights(scheme, _ptr(q_w), N, K, _ptr(q_w_packed), _stream(stream)), "qlin_pack_weights")


def qlin_linear_packed(scheme, x, segments, out=OUT_BF16, q_x=None, s_x=None, stream=None):
    """qlin_linear for M >= 33 with every segment's q_w [n, K] in the packed
    order that qlin_pack_weights writes (s_w and y as for qlin_linear);
    q_x / s_x staging required (s_x [M, K/128] for the block scheme)."""
    M, K = _dims2(x, "x", 2)
    _args(*_segment_args(scheme, M, K, segments, out), ("q_x", q_x, M * K, 1),
          ("s_x", s_x, 4 * _sx_count(scheme == SCHEME_FP8_BLOCK, M, K), 4), ("x", x, 0, None))
    arr = segments_array(segments)
    _check(_lib.qlin_linear_packed(scheme, _ptr(x), M, K, arr, len(segments), out, _ptr(q_x), _ptr(s_x),
                                   _stream(stream)), "qlin_linear_packed")


def qlin_linear_swiglu_packed(scheme, x, gate, up, h, q_x=None, s_x=None, stream=None):
    """qlin_linear_swiglu for M >= 33 with gate and up as (packed q_w [I, K],
    s_w) pairs from qlin_pack_weights; q_x / s_x staging required."""
    M, K = _dims2(x, "x", 2)
    (gq, gs), (uq, us) = gate, up
    if gq.dim() != 2 or gq.shape[1] != K or tuple(uq.shape) != tuple(gq.shape):
        raise ValueError("gate and up q_w must both be [I, K]")
    I = gq.shape[0]
    block = scheme == SCHEME_FP8_BLOCK
    _args(("gate q_w", gq, I * K, 1), ("up q_w", uq, I * K, 1), ("gate s_w", gs, 2 * _sw_count(block, I, K), 2),
          ("up s_w", us, 2 * _sw_count(block, I, K), 2), ("h", h, 2 * M * I, None), ("q_x", q_x, M * K, 1),
          ("s_x", s_x, 4 * _sx_count(block, M, K), 4), ("x", x, 0, None))
    _check(_lib.qlin_linear_swiglu_packed(scheme, _ptr(x), M, K, _ptr(gq), _ptr(gs), _ptr(uq), _ptr(us), I, _ptr(h),
                                          _ptr(q_x), _ptr(s_x), _stream(stream)), "qlin_linear_swiglu_packed")


def qlin_linear_noalloc(scheme, x, segments, out=OUT_BF16, stream=None):
    """qlin_linear with the library's fixed scratch as staging (no q_x / s_x):
    for callers that cannot allocate.  Calls that may overlap on one GPU race
    on the scratch."""
    M, K = _dims2(x, "x", 2)
    _args(*_segment_args(scheme, M, K, segments, out), ("x", x, 0, None))
    arr = segments_array(segments)
    _check(_lib.qlin_linear_noalloc(scheme, _ptr(x), M, K, arr, len(segments), out, _stream(stream)),
           "qlin_linear_noalloc")


def qlin_linear_weight_only(scheme, x, segments, out=OUT_BF16, stream=None):
    """Weight-only numerics: x bf16 [M, K] (M <= 32) times the dequantized
    weights of each segment (q_w [n, K], s_w, y [M, n]); the input is not rounded."""
    M, K = _dims2(x, "x", 2)
    _args(*_segment_args(scheme, M, K, segments, out), ("x", x, 0, None))
    arr = segments_array(segments)
    _check(_lib.qlin_linear_weight_only(scheme, _ptr(x), M, K, arr, len(segments), out, _stream(stream)),
           "qlin_linear_weight_only")


def qlin_linear_swiglu(scheme, x, gate, up, h, q_x=None, s_x=None, stream=None):
    """x bf16 [M, K]; gate, up: (q_w [I, K], s_w) of one gated MLP; h bf16
    [M, I] receives silu(gate projection) * (up projection), each rounded as
    the header states.  q_x / s_x: staging for the quantized activations
    (optional at M == 1)."""
    M, K = _dims2(x, "x", 2)
    (gq, gs), (uq, us) = gate, up
    if gq.dim() != 2 or gq.shape[1] != K or tuple(uq.shape) != tuple(gq.shape):
        raise ValueError("gate and up q_w must both be [I, K]")
    I = gq.shape[0]
    block = scheme == SCHEME_FP8_BLOCK
    _args(("gate q_w", gq, I * K, 1), ("up q_w", uq, I * K, 1), ("gate s_w", gs, 2 * _sw_count(block, I, K), 2),
          ("up s_w", us, 2 * _sw_count(block, I, K), 2), ("h", h, 2 * M * I, None), ("q_x", q_x, M * K, 1),
          ("s_x", s_x, 4 * _sx_count(block, M, K), 4), ("x", x, 0, None))
    _check(_lib.qlin_linear_swiglu(scheme, _ptr(x), M, K, _ptr(gq), _ptr(gs), _ptr(uq), _ptr(us), gq.shape[0],
                                   _ptr(h), _ptr(q_x), _ptr(s_x), _stream(stream)), "qlin_linear_swiglu")


# --------------------------------------------------------------------------
# 4-bit weights, routing and experts (include/qlin_w4.h)
#
# These calls run on the device of their first tensor, whichever device is
# current, on `stream` or that device's current stream.
# --------------------------------------------------------------------------

import torch as _torch  # noqa: E402  (loaded with the library above)


class W4Weight:
    """4-bit weights laid out for the library by qlin_pack_w4: one matrix
    [N, K], or `experts` of them.  Owns the packed tensors, which cannot be
    replaced (their contents can be written); copies and pickles hold tensors of
    their own."""

    def __init__(self, packed, scales, zeros, experts, N, K, group):
        # struct qlin_w4_weight as bytes: arrays of them are joined without building a ctypes object for each call
        vars(self).update(packed=packed, scales=scales, zeros=zeros, experts=experts, N=N, K=K, group=group, device=packed.device,
                          _bytes=bytes(QlinW4Weight(packed.data_ptr(), scales.data_ptr(), _ptr(zeros), N)))

    def __setattr__(self, name, value):
        raise AttributeError(f"{name} of a W4Weight cannot be replaced: pack the weights anew")

    def __reduce__(self):    # built again from the tensors: the addresses are theirs alone
        return W4Weight, (self.packed, self.scales, self.zeros, self.experts, self.N, self.K, self.group)


# Handle of a device's current stream, without building a Stream object where torch offers that.
_raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream",
                      lambda index: _torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)


def _launch(fn, device, stream, *args):
    if device.type != "cuda":
        raise ValueError("the tensors must be device tensors")
    index = device.index
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == _current_device():
        status = fn(*args, stream)
    else:
        with _torch.cuda.device(index):
            status = fn(*args, stream)
    if status != QLIN_OK:
        raise QlinError(status, fn.__name__)


# Types by element size; float16 is no type of theirs.
_TYPES = {size: frozenset(t for t in vars(_torch).values()
                          if isinstance(t, _torch.dtype) and t.itemsize == size and t is not _torch.float16) for size in (1, 2, 4)}


def _w4_tensor(t, name, shape, size, device):
    """One tensor argument of the calls below: exactly this shape (None: any), contiguous, on the call's device."""
    if t.dtype not in _TYPES[size] or (shape is not None and t.shape != shape) or not t.is_contiguous():
        if t.dtype is _torch.float16:
            raise ValueError(f"{name} must be bfloat16 (or its bit patterns), not float16")
        raise ValueError(f"{name} must be a contiguous tensor of {size}-byte elements"
                         + (f" and shape {list(shape)}, not {list(t.shape)}" if shape is not None else ""))
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")


def qlin_pack_w4(q_w, s_w, z_w=None):
    """q_w uint8 [N, K/2] (input 2 i in the low half of byte i) or [E, N, K/2],
    s_w bf16 [.., N, K/group], z_w uint8 like s_w or None (8) -> W4Weight.
    The packed weights are new tensors, written on the current stream; the arguments need not be kept."""
    if q_w.dim() not in (2, 3) or s_w.dim() != q_w.dim():
        raise ValueError("q_w must be [N, K/2] or [E, N, K/2], s_w [N, K/group] or [E, N, K/group]")
    E, N, K = (q_w.shape[0] if q_w.dim() == 3 else 1), q_w.shape[-2], 2 * q_w.shape[-1]
    groups = s_w.shape[-1]
    group = K // groups if groups else 0
    if group not in (32, 64, 128) or group * groups != K:
        raise ValueError(f"{groups} scales for {K} inputs: the group must be 32, 64 or 128 inputs")
    _w4_tensor(q_w, "q_w", None, 1, q_w.device)
    _w4_tensor(s_w, "s_w", (*q_w.shape[:-1], groups), 2, q_w.device)
    if z_w is not None:
        _w4_tensor(z_w, "z_w", (*q_w.shape[:-1], groups), 1, q_w.device)
    size = _lib.qlin_w4_packed_bytes(N, K)
    if (N and not size) or E > MAX_EXPERTS:
        raise QlinError(QLIN_ERR_SHAPE, "qlin_pack_w4")
    count = E * _lib.qlin_w4_packed_scales(N, K, group)
    packed = _torch.empty((E * size,), dtype=_torch.uint8, device=q_w.device)
    scales = _torch.empty((count,), dtype=s_w.dtype, device=q_w.device)
    zeros = None if z_w is None else _torch.empty((count,), dtype=z_w.dtype, device=q_w.device)
    _launch(_lib.qlin_pack_w4, q_w.device, None, q_w.data_ptr(), s_w.data_ptr(), _ptr(z_w), E, N, K, group, packed.data_ptr(),
            scales.data_ptr(), _ptr(zeros))
    return W4Weight(packed, scales, zeros, E, N, K, group)


def _w4_input(x):
    """-> (device, M, K) of the activations."""
    if x.dtype not in _TYPES[2] or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor of bfloat16 (or its bit patterns)")
    return x.device, *x.shape


def _w4_reads(w, name, K, device):
    if w.K != K or w.device != device:
        raise ValueError(f"{name} has {w.K} inputs on {w.device}, x {K} on {device}")


_POINTERS = [struct.Struct(f"{n}Q").pack for n in range(MAX_SEGMENTS + 1)]


def qlin_linear_w4(x, segments, out=OUT_BF16, stream=None):
    """x bf16 [M, K]; segments: list of (W4Weight [n, K], y [M, n]) sharing x, of one group size."""
    nw = len(segments)
    if not 1 <= nw <= MAX_SEGMENTS:
        raise ValueError(f"segments must hold one to {MAX_SEGMENTS} (weight, y) pairs")
    device, M, K = _w4_input(x)
    group, size = segments[0][0].group, _out_bytes(out)
    for w, y in segments:
        _w4_reads(w, "a segment", K, device)
        if w.experts != 1 or w.group != group:
            raise ValueError("every segment must be one matrix, all of one group size")
        _w4_tensor(y, "a segment's y", (M, w.N), size, device)
    weights = w._bytes if nw == 1 else b"".join([w._bytes for w, _ in segments])
    _launch(_lib.qlin_linear_w4, device, stream, x.data_ptr(), M, K, group, weights,
            _POINTERS[nw](*[y.data_ptr() for _, y in segments]), nw, out)


def qlin_linear_swiglu_w4(x, gate, up, h, stream=None):
    """x bf16 [M, K]; gate, up: W4Weight [I, K]; h bf16 [M, I] receives silu(x gate^T) * (x up^T), rounded once."""
    device, M, K = _w4_input(x)
    _w4_reads(gate, "gate", K, device)
    _w4_reads(up, "up", K, device)
    if gate.experts != 1 or up.experts != 1 or gate.N != up.N or gate.group != up.group:
        raise ValueError("gate and up must be one matrix each, of one shape and group size")
    _w4_tensor(h, "h", (M, gate.N), 2, device)
    _launch(_lib.qlin_linear_swiglu_w4, device, stream, x.data_ptr(), M, K, gate.group, gate._bytes, up._bytes, h.data_ptr())


def qlin_route(logits, ids, weights, score=SCORE_SOFTMAX, bias=None, groups=1, top_groups=1, group_best=2,
               renormalize=True, scale=1.0, stream=None):
    """logits bf16 or f32 [T, E]; ids int32 [T, k] and weights f32 [T, k] receive the k experts of each token."""
    dtype, device = logits.dtype, logits.device
    if (dtype is not _torch.float32 and dtype is not _torch.bfloat16) or logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous 2-D tensor of bfloat16 or float32")
    T, E = logits.shape
    if ids.dtype is not _torch.int32 or weights.dtype is not _torch.float32 or ids.dim() != 2:
        raise ValueError("ids must be int32 [T, k] and weights float32 [T, k]")
    shape = (T, ids.shape[1])
    _w4_tensor(ids, "ids", shape, 4, device)
    _w4_tensor(weights, "weights", shape, 4, device)
    if bias is not None:
        if bias.dtype is not _torch.float32:
            raise ValueError("bias must be float32 [E]")
        _w4_tensor(bias, "bias", (E,), 4, device)
    _launch(_lib.qlin_route, device, stream, logits.data_ptr(), OUT_F32 if dtype is _torch.float32 else OUT_BF16, T, E, shape[1],
            score, _ptr(bias), groups, top_groups, group_best, 1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr())


def qlin_experts_w4_workspace(T, k, gate, up, down):
    """Bytes of qlin_experts_w4's workspace for T tokens of k experts each."""
    size = _lib.qlin_experts_w4_workspace(T, k, gate.experts, gate.K, gate.N)
    if not size and T:
        raise QlinError(QLIN_ERR_SHAPE, "qlin_experts_w4_workspace")
    return size


def qlin_experts_w4(x, ids, weights, gate, up, down, y, workspace, stream=None):
    """x bf16 [T, H]; ids int32 [T, k] (outside 0..E-1: no expert), weights f32 [T, k]; gate, up: W4Weight of E
    matrices [I, H], down of E matrices [H, I]; y bf16 [T, H]; workspace uint8, qlin_experts_w4_workspace bytes."""
    device, T, H = _w4_input(x)
    _w4_reads(gate, "gate", H, device)
    E, I, group = gate.experts, gate.N, gate.group
    if (up.experts, up.N, up.K, up.group) != (E, I, H, group) or (down.experts, down.N, down.K, down.group) != (E, H, I, group):
        raise ValueError("up must have gate's shape, down be [E, H, I], all of one group size")
    if up.device != device or down.device != device:
        raise ValueError(f"every tensor must be on {device}")
    if ids.dim() != 2 or ids.dtype != _torch.int32 or weights.dtype != _torch.float32:
        raise ValueError("ids must be int32 [T, k] and weights float32 [T, k]")
    k = ids.shape[1]
    _w4_tensor(ids, "ids", (T, k), 4, device)
    _w4_tensor(weights, "weights", (T, k), 4, device)
    _w4_tensor(y, "y", (T, H), 2, device)
    _w4_tensor(workspace, "workspace", None, 1, device)
    need = _lib.qlin_experts_w4_workspace(T, k, E, H, I)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; the call needs {need}")
    _launch(_lib.qlin_experts_w4, device, stream, x.data_ptr(), T, H, I, E, k, group, ids.data_ptr(), weights.data_ptr(),
            gate._bytes, up._bytes, down._bytes, y.data_ptr(), workspace.data_ptr())


# --------------------------------------------------------------------------
# Between the projections of a layer (include/qlin_layer.h).  As the calls
# above, these run on the device of their first tensor.
# --------------------------------------------------------------------------

import math as _math  # noqa: E402


# Host time of a call weighs as much as a decode step's launch: these check a tensor in one go (its device by number) and
# say what is wrong only where something is.
_BYTE, _TWO = _TYPES[1], _TYPES[2]
_INT32, _FLOAT32 = frozenset([_torch.int32]), frozenset([_torch.float32])


def _expect(t, name, types, shape, index):
    """t is a contiguous tensor of this shape (None: any) and one of these types, on device number `index` (-1: the host)."""
    if t.dtype in types and (shape is None or t.shape == shape) and t.get_device() == index and t.is_contiguous():
        return
    if types is _INT32 or types is _FLOAT32:
        if t.dtype not in types:
            raise ValueError(f"{name} must be {'int32' if types is _INT32 else 'float32'}, not {t.dtype}")
    _w4_tensor(t, name, shape, {_BYTE: 1, _TWO: 2}.get(types, 4), t.device)
    raise ValueError(f"{name} is on {t.device}, the call runs on device {index}")


def _launch_on(fn, index, stream, *args):
    if index < 0:
        raise ValueError("the tensors must be device tensors")
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == _current_device():
        status = fn(*args, stream)
    else:
        with _torch.cuda.device(index):
            status = fn(*args, stream)
    if status != QLIN_OK:
        raise QlinError(status, fn.__name__)


def _norm(fn, x, gamma, outputs, group, residual, sum_out, eps, stream):
    """The three norms: outputs are (y,) or (q, s)."""
    if x.dtype not in _TWO or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor of bfloat16 (or its bit patterns)")
    index, shape = x.get_device(), x.shape
    M, K = shape
    _expect(gamma, "gamma", _TWO, (K,), index)
    if len(outputs) == 1:
        _expect(outputs[0], "y", _TWO, shape, index)
    else:
        _expect(outputs[0], "q", _BYTE, shape, index)
        _expect(outputs[1], "s", _FLOAT32, (M, K // 128) if group == 128 else (M,), index)
    if residual is not None and sum_out is not None:
        _expect(residual, "residual", _TWO, shape, index)
        if sum_out is not residual:
            _expect(sum_out, "sum_out", _TWO, shape, index)
        r, total = residual.data_ptr(), sum_out.data_ptr()
    elif residual is None and sum_out is None:
        r = total = None
    else:
        raise ValueError("residual and sum_out come together")
    more = () if group is None else (group,)
    _launch_on(fn, index, stream, x.data_ptr(), r, gamma.data_ptr(), M, K, eps, *more, total, *[t.data_ptr() for t in outputs])


def qlin_norm_bf16(x, gamma, y, residual=None, sum_out=None, eps=1e-6, stream=None):
    """x bf16 [M, K]; gamma bf16 [K]; y bf16 [M, K] receives the RMS norm of x, or of x + residual, which goes to
    sum_out (both bf16 [M, K]; sum_out may be residual itself)."""
    _norm(_lib.qlin_norm_bf16, x, gamma, (y,), None, residual, sum_out, eps, stream)


def qlin_norm_int8(x, gamma, q, s, residual=None, sum_out=None, eps=1e-6, stream=None):
    """qlin_norm_bf16 rounded for qlin_gemm_w8a8, in one launch: q int8 [M, K], s f32 [M]."""
    _norm(_lib.qlin_norm_int8, x, gamma, (q, s), None, residual, sum_out, eps, stream)


def qlin_norm_fp8(x, gamma, q, s, group=0, residual=None, sum_out=None, eps=1e-6, stream=None):
    """qlin_norm_bf16 rounded for qlin_gemm_fp8_*: q E4M3 codes [M, K], s f32 [M] (group 0) or [M, K/128] (group 128)."""
    _norm(_lib.qlin_norm_fp8, x, gamma, (q, s), group, residual, sum_out, eps, stream)


class _Fixed:
    """A description that holds device addresses: its tensors cannot be replaced (their contents can be written), and
    copies and pickles are built again from tensors of their own."""

    def __setattr__(self, name, value):
        raise AttributeError(f"{name} of a {type(self).__name__} cannot be replaced: build it anew")


class Rope(_Fixed):
    """Rotary positions of the first `dims` channels of a head: pair i turns by position * frequencies[i].

    frequencies: f64 [dims / 2], or None for base ** (-2 i / dims) with `scaling`
      "none";
      "linear": divided by factor;
      "ntk": of the base base * factor ** (dims / (dims - 2));
      "yarn": pairs that make `fast` (32) or more turns within the `original` length as they are, those that make
        `slow` (1) or fewer divided by factor, a ramp over the pairs between; strength 0.1 ln(factor) + 1;
      "bands": as they are from `fast` (4) turns on, divided by factor up to `slow` (1), between by the turns.
    interleaved: pairs are channels 2 i and 2 i + 1, else i and i + dims / 2.
    strength: factor of cosine and sine (1, or as above)."""

    def __init__(self, dims, base=10000.0, scaling="none", factor=1.0, original=None, interleaved=False, fast=None, slow=1.0,
                 strength=None, frequencies=None, device="cuda"):
        if dims < 16 or dims % 16 or dims > MAX_HEAD_DIM:
            raise ValueError(f"dims must be a multiple of 16 from 16 to {MAX_HEAD_DIM}, not {dims}")
        if frequencies is None:
            values, default = self._values(dims, base, scaling, factor, original, fast, slow)
            frequencies = _torch.tensor(values, dtype=_torch.float64, device=device)
        else:
            default = 1.0
        if frequencies.dtype is not _torch.float64 or frequencies.shape != (dims // 2,) or not frequencies.is_contiguous():
            raise ValueError(f"frequencies must be a contiguous float64 tensor of {dims // 2}")
        strength = default if strength is None else float(strength)
        vars(self).update(frequencies=frequencies, dims=dims, interleaved=bool(interleaved), strength=strength, device=frequencies.device, _index=frequencies.get_device(),
                          _bytes=bytes(QlinRotation(frequencies.data_ptr(), dims, 1 if interleaved else 0, strength)))

    @staticmethod
    def _values(dims, base, scaling, factor, original, fast, slow):
        if not (base > 1 and factor > 0 and _math.isfinite(base) and _math.isfinite(factor)):
            raise ValueError("base must be over 1 and factor over 0")
        if scaling == "ntk":
            base, factor, scaling = base * factor ** (dims / (dims - 2)), 1.0, "none"
        plain = [base ** (-2.0 * i / dims) for i in range(dims // 2)]
        if scaling == "none":
            return plain, 1.0
        if scaling == "linear":
            return [f / factor for f in plain], 1.0
        if scaling not in ("yarn", "bands"):
            raise ValueError(f"scaling must be none, linear, ntk, yarn or bands, not {scaling!r}")
        fast = (32.0 if scaling == "yarn" else 4.0) if fast is None else fast
        if original is None or not original > 0 or not fast > slow > 0:
            raise ValueError(f"{scaling} needs the original length, and fast over slow over 0")
        if scaling == "bands":
            stay = [(original * f / (2 * _math.pi) - slow) / (fast - slow) for f in plain]
            default = 1.0
        else:
            def pair(turns):   # the (fractional) pair that makes so many turns
                return dims * _math.log(original / (turns * 2 * _math.pi)) / (2 * _math.log(base))
            first = max(_math.floor(pair(fast)), 0)
            last = min(_math.ceil(pair(slow)), dims - 1)
            stay = [1 - (i - first) / max(last - first, 0.001) for i in range(dims // 2)]
            default = 0.1 * _math.log(factor) + 1 if factor > 1 else 1.0
        stay = [min(max(w, 0.0), 1.0) for w in stay]
        return [f * w + f / factor * (1 - w) for f, w in zip(plain, stay)], default

    def __reduce__(self):
        return _rope_again, (self.dims, self.interleaved, self.strength, self.frequencies)


def _rope_again(dims, interleaved, strength, frequencies):
    return Rope(dims, interleaved=interleaved, strength=strength, frequencies=frequencies)


_KINDS = {_torch.bfloat16: CACHE_BF16, _torch.int8: CACHE_INT8, _torch.uint8: CACHE_FP8, _torch.float8_e4m3fn: CACHE_FP8}


class KVCache(_Fixed):
    """The paged keys and values of one layer: k and v [pages, kv_heads, page_size, dim], bfloat16, int8 or E4M3
    (float8_e4m3fn or uint8 codes), the last two with k_scale and v_scale f32 [pages, kv_heads, page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.dtype not in _KINDS or v.dtype != k.dtype:
            raise ValueError("k and v must be [pages, kv_heads, page_size, dim] tensors of bfloat16, int8, float8_e4m3fn or uint8")
        kind, device, shape = _KINDS[k.dtype], k.device, tuple(k.shape)
        for name, t in (("k", k), ("v", v)):
            _w4_tensor(t, name, shape, 2 if kind == CACHE_BF16 else 1, device)
        if kind == CACHE_BF16:
            if k_scale is not None or v_scale is not None:
                raise ValueError("a bfloat16 cache has no scales")
        else:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t is None or t.dtype is not _torch.float32:
                    raise ValueError(f"{name} must be float32 [pages, kv_heads, page_size]")
                _w4_tensor(t, name, shape[:3], 4, device)
        pages, kv_heads, page_size, dim = shape
        if max(pages, kv_heads, page_size, dim) > 0x7fffffff:
            raise QlinError(QLIN_ERR_SHAPE, "KVCache")
        vars(self).update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, pages=pages, kv_heads=kv_heads, page_size=page_size, dim=dim, kind=kind,
                          device=device, _index=k.get_device(), _workspaces={}, _bytes=bytes(QlinKVCache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), pages, kv_heads,
                                                                  page_size, dim, kind)))

    @classmethod
    def empty(cls, pages, kv_heads, page_size, dim, dtype=_torch.float8_e4m3fn, device="cuda"):
        """A cache of zeros."""
        if dtype not in _KINDS:
            raise ValueError("dtype must be bfloat16, int8, float8_e4m3fn or uint8")
        shape = (pages, kv_heads, page_size, dim)
        k, v = (_torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        scales = () if _KINDS[dtype] == CACHE_BF16 else tuple(_torch.zeros(shape[:3], dtype=_torch.float32, device=device) for _ in range(2))
        return cls(k, v, *scales)

    def __reduce__(self):
        return KVCache, (self.k, self.v, self.k_scale, self.v_scale)


def _heads(t, name, T, heads, dim, index):
    """-> stride between the tokens of t, bf16 [T, heads, dim] with contiguous heads and any stride between tokens."""
    if t.dtype not in _TWO or t.dim() != 3 or t.get_device() != index:
        if t.dtype is _torch.float16:
            raise ValueError(f"{name} must be bfloat16 (or its bit patterns), not float16")
        raise ValueError(f"{name} must be a 3-D tensor of 2-byte elements on the call's device, not {t.dtype} {list(t.shape)} on {t.device}")
    if t.shape != (T, heads, dim):
        raise ValueError(f"{name} must be {[T, heads, dim]}, not {list(t.shape)}")
    between, inner, last = t.stride()
    if (last != 1 and dim > 1) or (inner != dim and heads > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return between if T > 1 else heads * dim


def _rope_bytes(rope, positions, T, index):
    _expect(positions, "positions", _INT32, (T,), index)
    if rope._index != index:
        raise ValueError(f"rope is on {rope.device}, the call runs on device {index}")
    return rope._bytes


def qlin_rope(x, positions, rope, y, gamma=None, eps=1e-6, stream=None):
    """x bf16 [T, heads, dim] (any stride between tokens); positions int32 [T]; y like x, may be x, receives the rotated
    heads.  gamma bf16 [dim]: each head's RMS norm first."""
    if x.dim() != 3:
        raise ValueError("x must be [T, heads, dim]")
    index = x.get_device()
    T, heads, dim = x.shape
    xs, ys = _heads(x, "x", T, heads, dim, index), _heads(y, "y", T, heads, dim, index)
    turn = _rope_bytes(rope, positions, T, index)
    if gamma is not None:
        _expect(gamma, "gamma", _TWO, (dim,), index)
    _launch_on(_lib.qlin_rope, index, stream, x.data_ptr(), xs, positions.data_ptr(), T, heads, dim, turn, _ptr(gamma), eps, y.data_ptr(), ys)


_PACK_QUERIES = struct.Struct("QqQQqi4x").pack


def qlin_cache_write(cache, slots, k, v, positions=None, rope=None, q=None, q_out=None, q_gamma=None, k_gamma=None, eps=1e-6, stream=None):
    """k, v bf16 [T, kv_heads, dim] (any stride between tokens) into slots int32 [T] of the cache (-1: not written), and
    q [T, heads, dim] into q_out (may be q), in one launch.  rope and positions int32 [T]: q and k are rotated;
    q_gamma, k_gamma bf16 [dim]: each head's RMS norm first."""
    index, dim, kv_heads = cache._index, cache.dim, cache.kv_heads
    T = slots.shape[0] if slots.dim() == 1 else -1
    _expect(slots, "slots", _INT32, (T,), index)
    ks, vs = _heads(k, "k", T, kv_heads, dim, index), _heads(v, "v", T, kv_heads, dim, index)
    turn = at = queries = None
    if rope is not None and positions is not None:
        turn, at = _rope_bytes(rope, positions, T, index), positions.data_ptr()
    elif rope is not None or positions is not None:
        raise ValueError("rope and positions come together")
    if k_gamma is not None:
        _expect(k_gamma, "k_gamma", _TWO, (dim,), index)
    if q is not None:
        if q.dim() != 3 or q_out is None or (rope is None and q_gamma is None):
            raise ValueError("q must be [T, heads, dim], with q_out, and rope or q_gamma")
        heads = q.shape[1]
        qs, os = _heads(q, "q", T, heads, dim, index), _heads(q_out, "q_out", T, heads, dim, index)
        if q_gamma is not None:
            _expect(q_gamma, "q_gamma", _TWO, (dim,), index)
        queries = _PACK_QUERIES(q.data_ptr(), qs, 0 if q_gamma is None else q_gamma.data_ptr(), q_out.data_ptr(), os, heads)
    elif q_out is not None or q_gamma is not None:
        raise ValueError("q_out and q_gamma need q")
    _launch_on(_lib.qlin_cache_write, index, stream, cache._bytes, slots.data_ptr(), T, k.data_ptr(), ks, v.data_ptr(), vs, at, turn,
               _ptr(k_gamma), eps, queries)


def qlin_cache_read(cache, slots, k, v, stream=None):
    """k, v bf16 [n, kv_heads, dim] receive the keys and values of slots int32 [n]; rows of a slot outside the cache stay."""
    index = cache._index
    n = slots.shape[0] if slots.dim() == 1 else -1
    _expect(slots, "slots", _INT32, (n,), index)
    shape = (n, cache.kv_heads, cache.dim)
    _expect(k, "k", _TWO, shape, index)
    _expect(v, "v", _TWO, shape, index)
    _launch_on(_lib.qlin_cache_read, index, stream, cache._bytes, slots.data_ptr(), n, k.data_ptr(), v.data_ptr())


def qlin_attn_decode_workspace(heads, cache):
    """Bytes of qlin_attn_decode's workspace, for any number of sequences and any lengths."""
    size = _lib.qlin_attn_decode_workspace(heads, cache.kv_heads, cache.dim)
    if not size:
        raise QlinError(QLIN_ERR_SHAPE, "qlin_attn_decode_workspace")
    return size


def qlin_attn_decode(q, cache, pages, lengths, out, workspace, scale=None, window=0, stream=None):
    """Attention of one new token per sequence: q, out bf16 [S, heads, dim]; pages int32 [S, columns], the pages of each
    sequence's tokens; lengths int32 [S] (0: out is zero, negative: left as it was); window > 0: the last tokens alone;
    scale: dim ** -0.5 unless given; workspace uint8, qlin_attn_decode_workspace bytes."""
    index, dim = cache._index, cache.dim
    if q.dim() != 3 or pages.dim() != 2:
        raise ValueError("q must be [S, heads, dim] and pages [S, columns]")
    S, heads, _ = q.shape
    shape = (S, heads, dim)
    columns = pages.shape[1]
    _expect(q, "q", _TWO, shape, index)
    _expect(out, "out", _TWO, shape, index)
    _expect(pages, "pages", _INT32, (S, columns), index)
    _expect(lengths, "lengths", _INT32, (S,), index)
    _expect(workspace, "workspace", _BYTE, None, index)
    need = cache._workspaces.get(heads)    # (a size by the number of heads: it goes by the shapes alone)
    if need is None:
        need = cache._workspaces[heads] = _lib.qlin_attn_decode_workspace(heads, cache.kv_heads, dim)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; the call needs {need}")
    _launch_on(_lib.qlin_attn_decode, index, stream, q.data_ptr(), cache._bytes, pages.data_ptr(), S, heads, columns, lengths.data_ptr(),
               window, dim ** -0.5 if scale is None else scale, out.data_ptr(), workspace.data_ptr())
