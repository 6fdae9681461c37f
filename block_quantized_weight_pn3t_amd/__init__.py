"""Python binding of libpn.so (C ABI in include/pn.h): PN (pn3t / pn4t) and NVFP4 W4A16
decode-step GEMV, validation, decode and quantizers, the microscaled key/value cache with the
attention that reads it, the verification of drafted tokens, and a prompt's norm, 8-bit products, keys
rotated into the cache and log probabilities, on MI355X (gfx950).

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
           "int8_quantize_rows", "add_norm", "gemm_int8_workspace_bytes", "gemm_int8", "cache_append",
           "logprobs_workspace_bytes", "logprobs",
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
ROW_MAX_WIDTH = 65536  # add_norm and int8_quantize_rows
GEMM_INT8_MAX_K = 131056
LOGPROBS_MAX_TOP = 64

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


class AddNormArgs(C.Structure):
    """pn_add_norm_args of include/pn.h."""
    _fields_ = [("type", C.c_int), ("weight_type", C.c_int), ("rows", C.c_int64), ("K", C.c_int64),
                ("x", C.c_void_p), ("x_stride", C.c_int64), ("residual", C.c_void_p),
                ("residual_stride", C.c_int64), ("sum", C.c_void_p), ("sum_stride", C.c_int64),
                ("weight", C.c_void_p), ("eps", C.c_float), ("out", C.c_void_p),
                ("out_stride", C.c_int64), ("codes", C.c_void_p), ("scales", C.c_void_p)]


class AppendArgs(C.Structure):
    """pn_append_args of include/pn.h."""
    _fields_ = [("type", C.c_int), ("Hq", C.c_int), ("q", C.c_void_p), ("q_token_stride", C.c_int64),
                ("q_head_stride", C.c_int64), ("q_out", C.c_void_p), ("q_out_token_stride", C.c_int64),
                ("q_out_head_stride", C.c_int64), ("k", C.c_void_p), ("k_token_stride", C.c_int64),
                ("k_head_stride", C.c_int64), ("v", C.c_void_p), ("v_token_stride", C.c_int64),
                ("v_head_stride", C.c_int64), ("rotation", C.c_void_p), ("rows", C.c_int64),
                ("rot", C.c_int), ("interleaved", C.c_int), ("positions", C.c_void_p),
                ("slots", C.c_void_p), ("T", C.c_int64)]


class LogprobsArgs(C.Structure):
    """pn_logprobs_args of include/pn.h."""
    _fields_ = [("type", C.c_int), ("top", C.c_int), ("R", C.c_int64), ("V", C.c_int64),
                ("stride", C.c_int64), ("logits", C.c_void_p), ("tokens", C.c_void_p),
                ("scale", C.c_float), ("logprob", C.c_void_p), ("rank", C.c_void_p),
                ("entropy", C.c_void_p), ("lse", C.c_void_p), ("top_ids", C.c_void_p),
                ("top_logprobs", C.c_void_p)]


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
    "pn_int8_quantize_rows": (_I32, [_I32, _P, _I64, _I64, _I64, _P, _P, _P]),
    "pn_add_norm": (_I32, [_P, _P]),
    "pn_gemm_int8_workspace_bytes": (_I64, [_I64, _I64, _I64]),
    "pn_gemm_int8_cut": (_I32, [_I64, _I64, _I64, _P]),
    "pn_gemm_int8": (_I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I32, _P, _I64, _P, _I64, _P]),
    "pn_cache_append": (_I32, [_P, _P, _P]),
    "pn_logprobs_workspace_bytes": (_I64, [_I64, _I64, _I32]),
    "pn_logprobs": (_I32, [_P, _P, _I64, _P]),
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
        cls.i32, cls.i64, cls.u8, cls.i8 = torch.int32, torch.int64, torch.uint8, torch.int8
        cls.kinds = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        cls.device = torch.cuda.current_device if torch.cuda.is_available() else lambda: None
        cls.raw_stream = lambda device: torch.cuda.current_stream().cuda_stream
        if torch.cuda.is_available() and hasattr(torch._C, "_cuda_getCurrentRawStream"):
            # the same without the objects in between, which take as long as a launch
            torch.cuda.init()
            cls.device, cls.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
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
    return T.raw_stream(T.device()) if stream is None else _stream(stream)


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
        self.pages, self.data, self.device = data.numel() // each, data, data.get_device()
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


# ---- a prompt's norm, 8-bit products, rotated keys, log probabilities -----------------------------
#
# As above; every tensor has to be on the current device, whose stream the call goes to.

def _misfit(t, name, dtype, shape, dev, how):
    """Says what is wrong with a tensor that is not what it has to be."""
    raise ValueError(f"{name} must be {how} of {dtype} {tuple(shape)} on the current device ({dev}), got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _flat(t, name, dtype, shape, dev):
    """The address of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _misfit(t, name, dtype, shape, dev, "a contiguous tensor")
    return t.data_ptr()


def _rows(t, name, dtype, shape, dev, written=False):
    """The spacing of the rows of t [rows, width]; rows that are written must not overlap."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _misfit(t, name, dtype, shape, dev, "rows")
    row, column = t.stride()
    if (column != 1 and shape[1] > 1) or (written and row < shape[1] and shape[0] > 1):
        _misfit(t, name, dtype, shape, dev, "contiguous rows" + " that do not overlap" * written)
    return row


def _plain(t, name, dim, dev, T):
    """The element type id and strides of a plain tensor of `dim` dimensions, the last of them contiguous."""
    kind = T.kinds.get(t.dtype)
    strides = t.stride()
    if kind is None or len(strides) != dim or t.get_device() != dev or (strides[-1] != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be a tensor of {dim} dimensions, the last contiguous, of float32, bfloat16 or "
                         f"float16 on the current device ({dev}), got {t.dtype} {tuple(t.shape)} with strides {strides} "
                         f"on {t.device}")
    return kind, strides


def _workspace(t, dev, T):
    """A workspace's address and bytes."""
    if t is None:
        return 0, 0
    n = t.numel()
    return _flat(t, "workspace", T.u8, (n,), dev), n


def int8_quantize_rows(x, codes, scales, stream=None):
    """codes int8[N, K] and scales fp32[N] <- the rows of x [N, K] as 8-bit integers with one scale each
    (pn_int8_quantize_rows): activations before gemm_int8, and its weights."""
    T = _names()
    dev = T.device()
    kind, (row, _) = _plain(x, "x", 2, dev, T)
    shape = n, k = x.shape
    codes_at, scales_at = _flat(codes, "codes", T.i8, shape, dev), _flat(scales, "scales", T.f32, (n,), dev)
    _check(_lib.pn_int8_quantize_rows(kind, x.data_ptr(), row, n, k, codes_at, scales_at, _handle(stream, T)),
           "pn_int8_quantize_rows")


_pack_add_norm = struct.Struct("@iiqqPqPqPqPfPqPP").pack  # pn_add_norm_args


def add_norm(x, weight, eps, out=None, codes=None, scales=None, residual=None, sum=None, stream=None):
    """The root-mean-square norm of x (+ residual) [N, K] with weight [K] (pn_add_norm): out [N, K] <- plain
    numbers of x's type, codes int8[N, K] and scales fp32[N] <- 8-bit rows for gemm_int8; either or both.
    sum [N, K] <- x + residual, which the norm is of; sum and out may be x or residual themselves."""
    T = _names()
    dev = T.device()
    kind, (x_row, _) = _plain(x, "x", 2, dev, T)
    shape = n, k = x.shape
    dt = x.dtype
    weight_kind = T.kinds.get(weight.dtype)
    if weight_kind is None:
        _misfit(weight, "weight", "a floating type", (k,), dev, "a contiguous tensor")
    weight_at = _flat(weight, "weight", weight.dtype, (k,), dev)
    residual_at = residual_row = sum_at = sum_row = out_at = out_row = codes_at = scales_at = 0
    if residual is not None:
        residual_row, residual_at = _rows(residual, "residual", dt, shape, dev), residual.data_ptr()
    if sum is not None:
        sum_row, sum_at = _rows(sum, "sum", dt, shape, dev, True), sum.data_ptr()
    if out is not None:
        out_row, out_at = _rows(out, "out", dt, shape, dev, True), out.data_ptr()
    if codes is not None or scales is not None:
        if codes is None or scales is None:
            raise ValueError("codes and scales go together")
        codes_at, scales_at = _flat(codes, "codes", T.i8, shape, dev), _flat(scales, "scales", T.f32, (n,), dev)
    elif out is None:
        raise ValueError("out, or codes and scales, must be given")
    a = _pack_add_norm(kind, weight_kind, n, k, x.data_ptr(), x_row, residual_at, residual_row, sum_at, sum_row,
                       weight_at, eps, out_at, out_row, codes_at, scales_at)
    _check(_lib.pn_add_norm(a, _handle(stream, T)), "pn_add_norm")


def gemm_int8_workspace_bytes(M, N, K):
    """Device bytes that gemm_int8 needs for a [M, K] and w [N, K]; enough for fewer rows of a, too."""
    return int(_lib.pn_gemm_int8_workspace_bytes(M, N, K))


def gemm_int8(a, a_scales, w, w_scales, out, workspace=None, stream=None):
    """out [M, N] (float32, bfloat16 or float16, rows of any spacing) <- the product of a int8[M, K] and w
    int8[N, K], rows scaled by a_scales fp32[M] and w_scales fp32[N] (pn_gemm_int8). workspace: a uint8
    tensor of gemm_int8_workspace_bytes."""
    T = _names()
    dev = T.device()
    kind, _ = _plain(out, "out", 2, dev, T)
    if a.dim() != 2 or w.dim() != 2:
        raise ValueError(f"a and w must be [M, K] and [N, K], got {tuple(a.shape)} and {tuple(w.shape)}")
    m, k = a.shape
    n = w.shape[0]
    a_at, w_at = _flat(a, "a", T.i8, (m, k), dev), _flat(w, "w", T.i8, (n, k), dev)
    a_scales_at = _flat(a_scales, "a_scales", T.f32, (m,), dev)
    w_scales_at = _flat(w_scales, "w_scales", T.f32, (n,), dev)
    row = _rows(out, "out", out.dtype, (m, n), dev, True)
    work_at, work_bytes = _workspace(workspace, dev, T)
    _check(_lib.pn_gemm_int8(a_at, a_scales_at, m, w_at, w_scales_at, n, k, kind, out.data_ptr(), row, work_at,
                             work_bytes, _handle(stream, T)), "pn_gemm_int8")


def _overlap(n, heads, dim, token, head):
    """Whether any of the dim numbers from t * token + h * head on belong to two (t < n, h < heads)."""
    if n == 0 or ((heads < 2 or head >= dim) and (n < 2 or token >= (heads - 1) * head + dim)):
        return False
    for h in range(heads):  # the two tokens nearest to the head's distance, which begins and ends inside the tensor
        t = h * head // token if token else 0
        for t in (min(t, n - 1), min(t + 1, n - 1)):
            if (t or h) and abs(t * token - h * head) < dim:
                return True
    return False


def _heads(t, name, dtype, shape, dev, written=False):
    """The token and head strides of t [T, heads, dim], channels contiguous; heads that are written must not overlap."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        token, head, channel = t.stride()
        if channel == 1 and not (written and _overlap(*shape, token, head)):
            return token, head
    _misfit(t, name, dtype, shape, dev, "a tensor with contiguous channels" + " and heads that do not overlap" * written)


_pack_append = struct.Struct("@iiPqqPqqPqqPqqPqiiPPq").pack  # pn_append_args


def cache_append(cache, k, v, slots, rotation, positions=None, q=None, q_out=None, interleaved=False, stream=None):
    """cache_write of k and v [T, heads, dim] with k turned by its tokens' positions, and q_out <- q
    [T, Hq, dim] turned likewise (q_out may be q) (pn_cache_append). rotation fp32 [P, rot]: the cosines and
    sines of each position for the first rot channels of a head; positions int64[T]: a token's row of it,
    its own number unless given. interleaved: channels (2j, 2j + 1) turn together, not (j, j + rot / 2)."""
    T = _names()
    dev = T.device()
    if cache.device != dev:
        raise ValueError(f"the cache must be on the current device ({dev}), got {cache.data.device}")
    kind, (k_token, k_head, _) = _plain(k, "k", 3, dev, T)
    n, dt = k.shape[0], k.dtype
    shape = (n, cache.heads, cache.dim)
    if k.shape != shape:
        _misfit(k, "k", dt, shape, dev, "a tensor")
    v_token, v_head = _heads(v, "v", dt, shape, dev)
    slots_at = _flat(slots, "slots", T.i64, (n,), dev)
    if rotation.dim() != 2:
        raise ValueError(f"rotation must be [positions, rot], got {tuple(rotation.shape)}")
    rows, rot = rotation.shape
    rotation_at = _flat(rotation, "rotation", T.f32, (rows, rot), dev)
    positions_at = hq = q_at = q_token = q_head = out_at = out_token = out_head = 0
    if positions is not None:
        positions_at = _flat(positions, "positions", T.i64, (n,), dev)
    if q is not None:
        if q.dim() != 3 or q_out is None:
            raise ValueError("q must be [T, Hq, dim], with q_out to go to")
        hq = q.shape[1]
        shape = (n, hq, cache.dim)
        q_token, q_head = _heads(q, "q", dt, shape, dev)
        out_token, out_head = _heads(q_out, "q_out", dt, shape, dev, True)
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    a = _pack_append(kind, hq, q_at, q_token, q_head, out_at, out_token, out_head, k.data_ptr(), k_token, k_head,
                     v.data_ptr(), v_token, v_head, rotation_at, rows, rot, 1 if interleaved else 0, positions_at,
                     slots_at, n)
    _check(_lib.pn_cache_append(cache.ref, a, _handle(stream, T)), "pn_cache_append")


def logprobs_workspace_bytes(R, V, top=0):
    """Device bytes that logprobs needs for R rows over V tokens and `top` likeliest tokens."""
    return int(_lib.pn_logprobs_workspace_bytes(R, V, top))


_pack_logprobs = struct.Struct("@iiqqqPPfPPPPPP").pack  # pn_logprobs_args


def logprobs(logits, tokens=None, logprob=None, workspace=None, rank=None, entropy=None, lse=None, top_ids=None,
             top_logprobs=None, scale=1.0, stream=None):
    """Rows of logits [R, V] as distributions (pn_logprobs). logprob fp32[R] <- the log probability of
    tokens int32[R], rank int32[R] <- how many tokens have a larger logit, entropy fp32[R], lse fp32[R] <- the
    log of the sum of exp(scale * logits), top_ids int32[R, top] and top_logprobs fp32[R, top] <- the likeliest
    tokens: those of them that are given. scale: at least V * 2^-121. workspace: a uint8 tensor of
    logprobs_workspace_bytes."""
    T = _names()
    dev = T.device()
    kind, (row, _) = _plain(logits, "logits", 2, dev, T)
    R, V = logits.shape
    one = (R,)
    tokens_at = logprob_at = rank_at = entropy_at = lse_at = ids_at = top_at = top = 0
    if tokens is not None:
        tokens_at = _flat(tokens, "tokens", T.i32, one, dev)
    elif logprob is not None or rank is not None:
        raise ValueError("logprob and rank need tokens")
    if logprob is not None:
        logprob_at = _flat(logprob, "logprob", T.f32, one, dev)
    if rank is not None:
        rank_at = _flat(rank, "rank", T.i32, one, dev)
    if entropy is not None:
        entropy_at = _flat(entropy, "entropy", T.f32, one, dev)
    if lse is not None:
        lse_at = _flat(lse, "lse", T.f32, one, dev)
    if top_ids is not None or top_logprobs is not None:
        if top_ids is None or top_logprobs is None or top_ids.dim() != 2:
            raise ValueError("top_ids and top_logprobs must both be [R, top]")
        top = top_ids.shape[1]
        ids_at = _flat(top_ids, "top_ids", T.i32, (R, top), dev)
        top_at = _flat(top_logprobs, "top_logprobs", T.f32, (R, top), dev)
    work_at, work_bytes = _workspace(workspace, dev, T)
    a = _pack_logprobs(kind, top, R, V, row, logits.data_ptr(), tokens_at, scale, logprob_at, rank_at, entropy_at,
                       lse_at, ids_at, top_at)
    _check(_lib.pn_logprobs(a, work_at, work_bytes, _handle(stream, T)), "pn_logprobs")
