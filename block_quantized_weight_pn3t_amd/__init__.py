"""Python binding of libpn.so (C ABI in include/pn.h): PN (pn3t / pn4t) and NVFP4 W4A16
decode-step GEMV, validation, decode and quantizers, the microscaled key/value cache with the
attention that reads it, and the verification of drafted tokens, on MI355X (gfx950).

Argument marshalling only: every step runs in the HIP kernels of libpn.so. PyTorch supplies device
memory and the current stream. There is no CPU fallback: if the library is missing, importing
this package raises ImportError; if a call fails, it raises PNError.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

__all__ = ["PN3T", "PN4T", "PNError", "row_bytes", "validate_rows", "validate_row",
           "dequantize_rows", "dequantize_row", "gemv", "gemv_group", "quantize_rows", "hadamard_rows",
           "gemv_hadamard", "gemv_hadamard_noalloc", "gemv_group_hadamard", "nvfp4_validate_rows",
           "nvfp4_dequantize_rows", "gemv_nvfp4", "fp8row_validate_rows", "fp8row_dequantize_rows", "gemv_fp8row",
           "MXFP8", "MXFP4", "Cache", "cache_page_bytes", "cache_write", "cache_read",
           "attend_workspace_bytes", "attend", "verify_workspace_bytes", "verify",
           "library_path", "status_string", "lib"]

PN3T = 124
PN4T = 125
GROUP = {PN3T: 80, PN4T: 64}
MAX_TOKENS = 4         # NVFP4 and row-scaled E4M3 GEMV
GEMV_MAX_TOKENS = 16   # PN GEMV
GEMV_HADAMARD_MAX_TOKENS = 4  # PN GEMV with the rotation fused
GEMV_GROUP_MAX_PARTS = 4  # matrices per pn_gemv_group call
NOALLOC_MAX_FLOATS = 262144  # M * K limit of pn_gemv_hadamard_noalloc
MXFP8 = 0              # cache formats
MXFP4 = 1
VERIFY_MAX_DRAFTS = 63

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libpn.so")

if not os.path.exists(library_path):
    raise ImportError(f"{library_path} is not built; run __graft_entry__.build() (hipcc, gfx950)")

_lib = C.CDLL(library_path)
_P, _I64, _I32, _F = C.c_void_p, C.c_int64, C.c_int, C.c_float


class GemvPart(C.Structure):
    """pn_gemv_part of include/pn.h: one matrix of a pn_gemv_group call."""
    _fields_ = [("type", C.c_int), ("W", C.c_void_p), ("N", C.c_int64), ("y", C.c_void_p)]


class CacheDesc(C.Structure):
    """pn_cache of include/pn.h."""
    _fields_ = [("format", C.c_int), ("heads", C.c_int), ("dim", C.c_int), ("page", C.c_int),
                ("pages", C.c_int64), ("data", C.c_void_p)]


class AttendArgs(C.Structure):
    """pn_attend_args of include/pn.h."""
    _fields_ = [("type", C.c_int), ("B", C.c_int), ("Q", C.c_int), ("Hq", C.c_int),
                ("q", C.c_void_p), ("q_seq_stride", C.c_int64), ("q_token_stride", C.c_int64),
                ("q_head_stride", C.c_int64), ("scale", C.c_float), ("table", C.c_void_p),
                ("table_stride", C.c_int64), ("table_width", C.c_int), ("lens", C.c_void_p),
                ("q_lens", C.c_void_p), ("prefix_table", C.c_void_p), ("prefix_len", C.c_int64),
                ("out", C.c_void_p), ("lse", C.c_void_p)]


_SIGS = {
    "pn_row_bytes": (_I64, [_I32, _I64]),
    "pn_status_string": (C.c_char_p, [_I32]),
    "pn_validate_rows": (_I32, [_I32, _P, _I64, _I64, _P, _P]),
    "pn_validate_row": (_I32, [_I32, _P, _I64, _P, _P]),
    "pn_dequantize_rows": (_I32, [_I32, _P, _I64, _I64, _P, _P]),
    "pn_dequantize_row": (_I32, [_I32, _P, _I64, _P, _P]),
    "pn_gemv": (_I32, [_I32, _P, _I64, _I64, _P, _I64, _P, _P]),
    "pn_gemv_group": (_I32, [C.POINTER(GemvPart), _I32, _I64, _P, _I64, _P]),
    "pn_gemv_group_hadamard": (_I32, [C.POINTER(GemvPart), _I32, _I64, _P, _I64, _I64, _P]),
    "pn_quantize_rows": (_I32, [_I32, _P, _I64, _I64, _P, _P, _P]),
    "pn_hadamard_rows": (_I32, [_P, _I64, _I64, _I64, _P, _P]),
    "pn_gemv_hadamard": (_I32, [_I32, _P, _I64, _I64, _P, _I64, _I64, _P, _P]),
    "pn_gemv_hadamard_noalloc": (_I32, [_I32, _P, _I64, _I64, _P, _I64, _I64, _P, _P]),
    "pn_nvfp4_validate_rows": (_I32, [_P, _F, _I64, _I64, _P, _P]),
    "pn_nvfp4_dequantize_rows": (_I32, [_P, _P, _F, _I64, _I64, _P, _P]),
    "pn_gemv_nvfp4": (_I32, [_P, _P, _F, _I64, _I64, _P, _I64, _P, _P]),
    "pn_fp8row_validate_rows": (_I32, [_P, _P, _I64, _I64, _P, _P]),
    "pn_fp8row_dequantize_rows": (_I32, [_P, _P, _I64, _I64, _P, _P]),
    "pn_gemv_fp8row": (_I32, [_P, _P, _I64, _I64, _P, _I64, _P, _P]),
    "pn_cache_page_bytes": (_I64, [_I32, _I32, _I32, _I32]),
    "pn_cache_write": (_I32, [_P, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P]),
    "pn_cache_read": (_I32, [_P, _I32, _P, _I64, _P, _P, _P]),
    "pn_attend_workspace_bytes": (_I64, [_P, _P]),
    "pn_attend": (_I32, [_P, _P, _P, _I64, _P]),
    "pn_verify_workspace_bytes": (_I64, [_I64, _I64]),
    "pn_verify": (_I32, [_I32, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P,
                         _I64, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib() -> C.CDLL:
    return _lib


class PNError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def status_string(status: int) -> str:
    return _lib.pn_status_string(status).decode()


def _check(status: int, what: str):
    if status != 0:
        raise PNError(status, what)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


def _dev(t, name, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def row_bytes(type_: int, K: int) -> int:
    return int(_lib.pn_row_bytes(type_, K))


# ---- PN ---------------------------------------------------------------------------------------

def validate_rows(type_, W, nrows, K, verdict, stream=None):
    """verdict (int32[nrows], device) <- 1 valid / 0 invalid per row."""
    import torch
    _dev(verdict, "verdict", torch.int32)
    _check(_lib.pn_validate_rows(type_, _ptr(W), nrows, K, _ptr(verdict), _stream(stream)),
           "pn_validate_rows")


def validate_row(type_, row, K, verdict, stream=None):
    _check(_lib.pn_validate_row(type_, _ptr(row), K, _ptr(verdict), _stream(stream)),
           "pn_validate_row")


def dequantize_rows(type_, W, nrows, K, out, stream=None):
    import torch
    _dev(out, "out", torch.float32)
    _check(_lib.pn_dequantize_rows(type_, _ptr(W), nrows, K, _ptr(out), _stream(stream)),
           "pn_dequantize_rows")


def dequantize_row(type_, row, K, out, stream=None):
    _check(_lib.pn_dequantize_row(type_, _ptr(row), K, _ptr(out), _stream(stream)),
           "pn_dequantize_row")


def gemv(type_, W, N, K, x, y, M=None, stream=None):
    """y[M, N] <- W[N, K] . x[M, K]^T for PN weights W (raw bytes on the device)."""
    import torch
    _dev(x, "x", torch.float32)
    _dev(y, "y", torch.float32)
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    _check(_lib.pn_gemv(type_, _ptr(W), N, K, _ptr(x), M, _ptr(y), _stream(stream)), "pn_gemv")


def gemv_group(parts, K, x, M=None, stream=None):
    """Several PN GEMVs that share x: parts is a sequence of (type, W, N, y) with W raw PN bytes
    and y fp32[M, N] on the device; every y[M, N] <- W[N, K] . x[M, K]^T, in one launch where the
    shapes allow (pn_gemv_group)."""
    import torch
    _dev(x, "x", torch.float32)
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    arr = (GemvPart * len(parts))()
    for i, (type_, W, N, y) in enumerate(parts):
        _dev(y, "y", torch.float32)
        arr[i] = GemvPart(type_, _ptr(W), N, _ptr(y))
    _check(_lib.pn_gemv_group(arr, len(parts), K, _ptr(x), M, _stream(stream)), "pn_gemv_group")


def gemv_group_hadamard(parts, K, x, B, M=None, stream=None):
    """gemv_group over x rotated in slices of B (pn_gemv_group_hadamard); x is not modified."""
    import torch
    _dev(x, "x", torch.float32)
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    arr = (GemvPart * len(parts))()
    for i, (type_, W, N, y) in enumerate(parts):
        _dev(y, "y", torch.float32)
        arr[i] = GemvPart(type_, _ptr(W), N, _ptr(y))
    _check(_lib.pn_gemv_group_hadamard(arr, len(parts), K, _ptr(x), M, B, _stream(stream)),
           "pn_gemv_group_hadamard")


def gemv_group_hadamard_ptr(parts, K, x_ptr, M, B, stream_handle):
    """Raw-pointer form: parts a prepared GemvPart array; returns the status."""
    return _lib.pn_gemv_group_hadamard(parts, len(parts), K, x_ptr, M, B, stream_handle)


def gemv_group_ptr(parts, K, x_ptr, M, stream_handle):
    """Raw-pointer form for timing loops: parts is a sequence of (type, W_ptr, N, y_ptr) or a
    prepared GemvPart array; returns the status instead of raising."""
    if not isinstance(parts, C.Array):
        arr = (GemvPart * len(parts))()
        for i, (type_, W, N, y) in enumerate(parts):
            arr[i] = GemvPart(type_, W, N, y)
        parts = arr
    return _lib.pn_gemv_group(parts, len(parts), K, x_ptr, M, stream_handle)


def gemv_ptr(type_, W_ptr, N, K, x_ptr, M, y_ptr, stream_handle):
    """Raw-pointer form for timing loops: returns the status instead of raising."""
    return _lib.pn_gemv(type_, W_ptr, N, K, x_ptr, M, y_ptr, stream_handle)


def hadamard_rows(x, B, out, M=None, K=None, stream=None):
    """out[M, K] <- x rotated by the orthonormal Walsh-Hadamard matrix on slices of B elements."""
    import torch
    _dev(x, "x", torch.float32)
    _dev(out, "out", torch.float32)
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    if K is None:
        K = x.shape[-1]
    _check(_lib.pn_hadamard_rows(_ptr(x), M, K, B, _ptr(out), _stream(stream)), "pn_hadamard_rows")


def gemv_hadamard(type_, W, N, K, x, B, y, M=None, stream=None):
    """y[M, N] <- W[N, K] . (H x)[M, K]^T: x rotated into the library's per-device workspace, then
    the GEMV (M <= 4)."""
    import torch
    _dev(x, "x", torch.float32)
    _dev(y, "y", torch.float32)
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    _check(_lib.pn_gemv_hadamard(type_, _ptr(W), N, K, _ptr(x), M, B, _ptr(y), _stream(stream)),
           "pn_gemv_hadamard")


def gemv_hadamard_noalloc(type_, W, N, K, x, B, y, M=None, stream=None):
    """As gemv_hadamard, with the rotated x in the library's own device array (no allocation;
    M * K <= PN_NOALLOC_MAX_FLOATS; calls that overlap on one GPU race on that array)."""
    import torch
    _dev(x, "x", torch.float32)
    _dev(y, "y", torch.float32)
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    _check(_lib.pn_gemv_hadamard_noalloc(type_, _ptr(W), N, K, _ptr(x), M, B, _ptr(y),
                                         _stream(stream)), "pn_gemv_hadamard_noalloc")


def gemv_hadamard_ptr(type_, W_ptr, N, K, x_ptr, M, B, y_ptr, stream_handle):
    """Raw-pointer form for timing loops: returns the status instead of raising."""
    return _lib.pn_gemv_hadamard(type_, W_ptr, N, K, x_ptr, M, B, y_ptr, stream_handle)


def quantize_rows(type_, w, W, status=None, stream=None):
    """PN reference quantizer: W (uint8[nrows, row_bytes], device) <- fp32 w[nrows, K]."""
    import torch
    _dev(w, "w", torch.float32)
    nrows, K = w.shape
    _check(_lib.pn_quantize_rows(type_, _ptr(w), nrows, K, _ptr(W), _ptr(status),
                                 _stream(stream)), "pn_quantize_rows")


# ---- NVFP4 ------------------------------------------------------------------------------------

def nvfp4_validate_rows(scales, g, N, K, verdict, stream=None):
    _check(_lib.pn_nvfp4_validate_rows(_ptr(scales), g, N, K, _ptr(verdict), _stream(stream)),
           "pn_nvfp4_validate_rows")


def nvfp4_dequantize_rows(codes, scales, g, N, K, out, stream=None):
    _check(_lib.pn_nvfp4_dequantize_rows(_ptr(codes), _ptr(scales), g, N, K, _ptr(out),
                                         _stream(stream)), "pn_nvfp4_dequantize_rows")


def gemv_nvfp4(codes, scales, g, N, K, x_bf16, y, M=None, stream=None):
    """y[M, N] <- NVFP4 W . x; x_bf16 holds raw bf16 words (int16/uint16/bfloat16 tensor)."""
    if M is None:
        M = 1 if x_bf16.dim() == 1 else x_bf16.shape[0]
    _check(_lib.pn_gemv_nvfp4(_ptr(codes), _ptr(scales), g, N, K, _ptr(x_bf16), M, _ptr(y),
                              _stream(stream)), "pn_gemv_nvfp4")


def gemv_nvfp4_ptr(codes_ptr, scales_ptr, g, N, K, x_ptr, M, y_ptr, stream_handle):
    return _lib.pn_gemv_nvfp4(codes_ptr, scales_ptr, g, N, K, x_ptr, M, y_ptr, stream_handle)


# ---- row-scaled E4M3FN (FP8_E4M3FN_ROW_BF16S) ----------------------------------------------------

def fp8row_validate_rows(codes, scales, N, K, verdict, stream=None):
    _check(_lib.pn_fp8row_validate_rows(_ptr(codes), _ptr(scales), N, K, _ptr(verdict),
                                        _stream(stream)), "pn_fp8row_validate_rows")


def fp8row_dequantize_rows(codes, scales, N, K, out, stream=None):
    _check(_lib.pn_fp8row_dequantize_rows(_ptr(codes), _ptr(scales), N, K, _ptr(out),
                                          _stream(stream)), "pn_fp8row_dequantize_rows")


def gemv_fp8row(codes, scales, N, K, x, y, M=None, stream=None):
    """y[M, N] <- (row-scaled E4M3) W . x, x fp32[M, K]."""
    if M is None:
        M = 1 if x.dim() == 1 else x.shape[0]
    _check(_lib.pn_gemv_fp8row(_ptr(codes), _ptr(scales), N, K, _ptr(x), M, _ptr(y),
                               _stream(stream)), "pn_gemv_fp8row")


def gemv_fp8row_ptr(codes_ptr, scales_ptr, N, K, x_ptr, M, y_ptr, stream_handle):
    return _lib.pn_gemv_fp8row(codes_ptr, scales_ptr, N, K, x_ptr, M, y_ptr, stream_handle)


# ---- microscaled cache, attention over it, verification of drafts ---------------------------------
#
# A decode step makes these calls one after another while each kernel runs for a few microseconds, so
# a call's checks are single expressions that hold for good arguments; what is wrong with bad ones is
# worked out afterwards.

class _Torch:
    """torch's names that the checks below use, looked up once."""
    f32 = None

    @classmethod
    def load(cls):
        import torch
        cls.i32, cls.i64, cls.u8 = torch.int32, torch.int64, torch.uint8
        cls.kinds = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        cls.stream = torch.cuda.current_stream
        cls.f32 = torch.float32
        return cls


def _names():
    return _Torch if _Torch.f32 is not None else _Torch.load()


def _is(t, dtype, shape):
    return t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _refuse(t, name, dtype, shape):
    """Says what is wrong with a tensor that _is() not what it has to be."""
    _dev(t, name, dtype)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _elem(t, name, T):
    """The element type id of a plain tensor on the device."""
    kind = T.kinds.get(t.dtype)
    if kind is None or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor of float32, bfloat16 or float16, got {t.dtype} "
                         f"on {t.device}")
    return kind


def _handle(stream, T):
    return T.stream().cuda_stream if stream is None else _stream(stream)


def cache_page_bytes(format, heads, dim, page):
    """Bytes of one page of a cache (pn_cache_page_bytes); 0 where the library has no such cache."""
    return int(_lib.pn_cache_page_bytes(format, heads, dim, page))


class Cache:
    """A paged microscaled key/value cache over `data`, a contiguous uint8 device tensor of whole pages
    (cache_page_bytes each). Token places are slots: page number * page + place in the page. The bytes
    need no initial value: only tokens that were written are ever used."""

    def __init__(self, format, heads, dim, page, data):
        import torch
        each = cache_page_bytes(format, heads, dim, page)
        if each == 0:
            raise ValueError(f"no cache of format {format} with {heads} heads of {dim} channels and "
                             f"pages of {page} tokens")
        _dev(data, "data", torch.uint8)
        if data.numel() % each:
            raise ValueError(f"data must be whole pages of {each} bytes, got {data.numel()}")
        self.format, self.heads, self.dim, self.page = format, heads, dim, page
        self.pages, self.data = data.numel() // each, data
        self.desc = CacheDesc(format, heads, dim, page, self.pages, data.data_ptr())
        self.ref = C.addressof(self.desc)


def cache_write(cache, k, v, slots, stream=None):
    """Quantises k and v [T, heads, dim] (channels contiguous) into the cache; token t goes to
    slots[t] (int64), nowhere where that is outside the cache (pn_cache_write)."""
    T = _names()
    kind = _elem(k, "k", T)
    n = k.shape[0]
    shape = (n, cache.heads, cache.dim)
    kt, kh, kc = k.stride() if k.shape == shape else (0, 0, 0)
    vt, vh, vc = v.stride() if v.shape == shape else (0, 0, 0)
    if kc != 1 or vc != 1:
        raise ValueError(f"k and v must have shape {shape} with contiguous channels, got "
                         f"{tuple(k.shape)} and {tuple(v.shape)} with strides {k.stride()}, {v.stride()}")
    if v.dtype is not k.dtype or not v.is_cuda:
        raise ValueError("k and v must have the same type and be on the device")
    if not _is(slots, T.i64, (n,)):
        _refuse(slots, "slots", T.i64, (n,))
    _check(_lib.pn_cache_write(cache.ref, kind, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                               slots.data_ptr(), n, _handle(stream, T)), "pn_cache_write")


def cache_read(cache, slots, k, v, stream=None):
    """k and v [T, heads, dim] <- the cache's tokens at slots (int64); zeros for a slot outside it
    (pn_cache_read)."""
    T = _names()
    kind = _elem(k, "k", T)
    n = k.shape[0]
    shape = (n, cache.heads, cache.dim)
    if not _is(k, k.dtype, shape):
        _refuse(k, "k", k.dtype, shape)
    if not _is(v, k.dtype, shape):
        _refuse(v, "v", k.dtype, shape)
    if not _is(slots, T.i64, (n,)):
        _refuse(slots, "slots", T.i64, (n,))
    _check(_lib.pn_cache_read(cache.ref, kind, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(),
                              _handle(stream, T)), "pn_cache_read")


def attend_workspace_bytes(cache, q, table, prefix_len=0):
    """Device bytes that attend needs for q [B, Q, Hq, dim] and these tables."""
    B, Q, Hq, _ = q.shape
    a = AttendArgs(type=_elem(q, "q", _names()), B=B, Q=Q, Hq=Hq, scale=1.0, table_width=table.shape[1],
                   prefix_len=prefix_len)
    return int(_lib.pn_attend_workspace_bytes(cache.ref, C.addressof(a)))


_pack_attend = struct.Struct("@iiiiPqqqfPqiPPPqPP").pack  # pn_attend_args, a third of AttendArgs()'s time


def attend(cache, q, table, lens, out, lse=None, workspace=None, prefix_table=None, prefix_len=0,
           q_lens=None, scale=None, stream=None):
    """out [B, Q, Hq, dim] <- attention of q [B, Q, Hq, dim] (any strides, channels contiguous) over the
    first prefix_len tokens of the pages in prefix_table (int32), which every sequence sees, and over
    each sequence's own tokens: lens int32[B], in the pages of table int32[B, width] (pn_attend). The
    last of the own tokens are the queries', each sees up to itself. lse fp32[B, Q, Hq] <- the log of
    the sum of exp(scores). q_lens int32[B]: query tokens that a sequence has, Q unless given. scale:
    dim ** -0.5 unless given. workspace: a uint8 tensor of attend_workspace_bytes."""
    T = _names()
    kind = _elem(q, "q", T)
    if q.dim() != 4 or q.shape[3] != cache.dim:
        raise ValueError(f"q must be [B, Q, Hq, {cache.dim}], got {tuple(q.shape)}")
    B, Q, Hq, dim = shape = q.shape
    qb, qt, qh, qc = q.stride()
    if qc != 1:
        raise ValueError("the channels of q must be contiguous")
    if table.dim() != 2 or table.shape[0] != B or table.dtype is not T.i32 or not table.is_cuda:
        raise ValueError(f"table must be an int32 device tensor [{B}, width], got {table.dtype} "
                         f"{tuple(table.shape)} on {table.device}")
    width = table.shape[1]
    row, column = table.stride()
    if column != 1 and width > 1:
        raise ValueError("the rows of table must be contiguous")
    if not _is(lens, T.i32, (B,)):
        _refuse(lens, "lens", T.i32, (B,))
    if not _is(out, q.dtype, shape):
        _refuse(out, "out", q.dtype, shape)
    lse_at = q_lens_at = prefix_at = work_at = work_bytes = 0
    if lse is not None:
        if not _is(lse, T.f32, (B, Q, Hq)):
            _refuse(lse, "lse", T.f32, (B, Q, Hq))
        lse_at = lse.data_ptr()
    if q_lens is not None:
        if not _is(q_lens, T.i32, (B,)):
            _refuse(q_lens, "q_lens", T.i32, (B,))
        q_lens_at = q_lens.data_ptr()
    if prefix_len < 0:
        raise ValueError("prefix_len must not be negative")
    if prefix_len:
        _dev(prefix_table, "prefix_table", T.i32)
        if prefix_table.numel() * cache.page < prefix_len:
            raise ValueError("prefix_table has too few pages for prefix_len")
        prefix_at = prefix_table.data_ptr()
    if workspace is not None:
        _dev(workspace, "workspace", T.u8)
        work_at, work_bytes = workspace.data_ptr(), workspace.numel()
    a = _pack_attend(kind, B, Q, Hq, q.data_ptr(), qb, qt, qh, dim ** -0.5 if scale is None else scale,
                     table.data_ptr(), row, width, lens.data_ptr(), q_lens_at, prefix_at, prefix_len,
                     out.data_ptr(), lse_at)
    _check(_lib.pn_attend(cache.ref, a, work_at, work_bytes, _handle(stream, T)), "pn_attend")


def verify_workspace_bytes(B, V):
    """Device bytes that verify needs for B sequences over V tokens."""
    return int(_lib.pn_verify_workspace_bytes(B, V))


def _row_spacing(t, name, n):
    """The spacing of the n rows a sequence that t [B, n, V] has."""
    b, row, v = t.stride()
    if (v != 1 and t.shape[2] > 1) or (t.shape[0] > 1 and n > 1 and b != n * row):
        raise ValueError(f"the rows of {name} must be contiguous and evenly spaced")
    return row if n > 1 else b


def verify(p, q, draft, u_accept, u_sample, tokens, accepted, workspace, n_draft=None, stream=None):
    """Drafted tokens against the target's probabilities (pn_verify): p [B, K + 1, V] the target's, q
    [B, K, V] the draft's (None where each draft was certain), rows of any even spacing; draft
    int32[B, K], u_accept fp32[B, K] and u_sample fp32[B] random numbers in [0, 1); tokens
    int32[B, K + 1] <- the accepted drafts, the token after them, then -1; accepted int32[B] <- their
    number. n_draft int32[B]: drafts that a sequence has, K unless given. workspace: a uint8 tensor
    of verify_workspace_bytes."""
    T = _names()
    kind = _elem(p, "p", T)
    if draft.dim() != 2:
        raise ValueError(f"draft must be [B, K], got {tuple(draft.shape)}")
    B, K = shape = draft.shape
    if p.dim() != 3 or p.shape[0] != B or p.shape[1] != K + 1:
        raise ValueError(f"p must be [{B}, {K + 1}, V], got {tuple(p.shape)}")
    V = p.shape[2]
    p_row, q_row, q_at, n_at = _row_spacing(p, "p", K + 1), 0, 0, 0
    if q is not None:
        if q.dtype is not p.dtype or q.shape != (B, K, V) or not q.is_cuda:
            raise ValueError(f"q must be a device tensor of {p.dtype} [{B}, {K}, {V}], got {q.dtype} "
                             f"{tuple(q.shape)} on {q.device}")
        if K:
            q_row, q_at = _row_spacing(q, "q", K), q.data_ptr()
    if not _is(draft, T.i32, shape):
        _refuse(draft, "draft", T.i32, shape)
    if not _is(u_accept, T.f32, shape):
        _refuse(u_accept, "u_accept", T.f32, shape)
    if not _is(u_sample, T.f32, (B,)):
        _refuse(u_sample, "u_sample", T.f32, (B,))
    if not _is(tokens, T.i32, (B, K + 1)):
        _refuse(tokens, "tokens", T.i32, (B, K + 1))
    if not _is(accepted, T.i32, (B,)):
        _refuse(accepted, "accepted", T.i32, (B,))
    if n_draft is not None:
        if not _is(n_draft, T.i32, (B,)):
            _refuse(n_draft, "n_draft", T.i32, (B,))
        n_at = n_draft.data_ptr()
    _dev(workspace, "workspace", T.u8)
    _check(_lib.pn_verify(kind, p.data_ptr(), p_row, q_at, q_row, draft.data_ptr(), n_at,
                          u_accept.data_ptr(), u_sample.data_ptr(), B, K, V, tokens.data_ptr(),
                          accepted.data_ptr(), workspace.data_ptr(), workspace.numel(),
                          _handle(stream, T)), "pn_verify")
