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
ABI_VERSION = 4
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
    for name, (res, args) in {**SIGNATURES, **SIGNATURES_W4}.items():
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
