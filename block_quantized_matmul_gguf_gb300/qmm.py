"""Thin ctypes binding of libqmm.so (include/qmm.h), same entry-point names.

Only argument marshalling happens here: tensors become device pointers and
the stream becomes the current torch CUDA stream unless one is given.  Every
step of the computation runs in the library's CUDA kernels.  There is no
fallback: if libqmm.so cannot be loaded, every call raises.

Each function takes torch CUDA tensors (or raw integer device pointers) and
raises :class:`QmmError` when the library returns a non-OK status.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import build as _build

QMM_OK = 0
QMM_ERR_NULL = 1
QMM_ERR_SHAPE = 2
QMM_ERR_ALIGN = 3
QMM_ERR_UNSUPPORTED = 4
QMM_ERR_CUDA = 5
QMM_ERR_TIMEOUT = 6
QMM_ERR_SCRATCH = 7
QMM_ERR_INDEX = 8
QMM_F32 = 0
QMM_BF16 = 1
QMM_GEMV_MAX_M = 16

QMM_GEMV_MAX_OUTPUTS = 4

EXPORTED = (
    "qmm_dequant_q4_0", "qmm_dequant_q8_0", "qmm_gemv_q4_0", "qmm_gemv_q8_0",
    "qmm_gemv_q4_0_multi", "qmm_gemv_q8_0_multi", "qmm_gemv_q4_0_geglu", "qmm_gemv_q4_0_tc",
    "qmm_gemm_q4_0", "qmm_gemm_q8_0", "qmm_gemm_q4_0_geglu",
    "qmm_gemm_q4_0_ws", "qmm_gemm_q8_0_ws", "qmm_gemm_q4_0_geglu_ws", "qmm_gemm_q4_0_prefill",
    "qmm_gemm_workspace_bytes", "qmm_gemm_geglu_workspace_bytes", "qmm_status_string", "qmm_version", "qmm_get_device_error",
    "qmm_set_wait_timeout_ns", "qmm_selftest_wait_timeout", "qmm_copy",
    "qmm_kv_plan", "qmm_kv_append_q4_0", "qmm_kv_read_q4_0",
    "qmm_attn_q4_0_workspace_bytes", "qmm_attn_q4_0", "qmm_logits_adjust",
)


class GemvOut(ctypes.Structure):
    """struct qmm_gemv_out: one weight matrix and its output."""
    _fields_ = [("w", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n", ctypes.c_int64)]


class KvQ4_0(ctypes.Structure):
    """struct qmm_kv_q4_0: the arrays and sizes of a paged Q4_0 cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class AttnArgs(ctypes.Structure):
    """struct qmm_attn_args."""
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("q_type", ctypes.c_int),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("out_type", ctypes.c_int),
                ("lse", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_width", ctypes.c_int64),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("batch", ctypes.c_int),
                ("total_q", ctypes.c_int64), ("max_q", ctypes.c_int), ("heads", ctypes.c_int),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("window", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class LogitsArgs(ctypes.Structure):
    """struct qmm_logits_args."""
    _fields_ = [("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("history", ctypes.c_void_p), ("hist_start", ctypes.c_void_p),
                ("history_len", ctypes.c_int64), ("prompt_len", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
                ("bias_values", ctypes.c_void_p), ("bias_start", ctypes.c_void_p),
                ("bias_len", ctypes.c_int64), ("allowed", ctypes.c_void_p)]


class QmmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libqmm.so (building it first if asked and it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if not os.path.exists(path):
        if not build_if_missing:
            raise OSError(f"libqmm.so not built at {path}")
        _build.build_library()
    lib = ctypes.CDLL(path)
    P, I64, I32, U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
    SZ = ctypes.c_size_t
    sig = {
        "qmm_dequant_q4_0": [P, P, I64, I64, P],
        "qmm_dequant_q8_0": [P, P, I64, I64, P],
        "qmm_gemv_q4_0": [P, P, P, I32, I64, I64, P],
        "qmm_gemv_q8_0": [P, P, P, I32, I64, I64, P],
        "qmm_gemv_q4_0_tc": [P, P, P, I32, I64, I64, P],
        "qmm_gemm_q4_0": [P, P, P, I64, I64, I64, P],
        "qmm_gemm_q8_0": [P, P, P, I64, I64, I64, P],
        "qmm_gemv_q4_0_geglu": [P, P, P, P, I32, I64, I64, P],
        "qmm_gemm_q4_0_geglu": [P, P, P, P, I64, I64, I64, P],
        "qmm_gemm_q4_0_ws": [P, P, P, I64, I64, I64, P, SZ, P],
        "qmm_gemm_q4_0_prefill": [P, P, P, I64, I64, I64, P],
        "qmm_gemm_q8_0_ws": [P, P, P, I64, I64, I64, P, SZ, P],
        "qmm_gemm_q4_0_geglu_ws": [P, P, P, P, I64, I64, I64, P, SZ, P],
        "qmm_gemv_q4_0_multi": [ctypes.POINTER(GemvOut), I32, P, I32, I64, P],
        "qmm_gemv_q8_0_multi": [ctypes.POINTER(GemvOut), I32, P, I32, I64, P],
        "qmm_get_device_error": [P],
        "qmm_selftest_wait_timeout": [U64, P],
        "qmm_copy": [P, P, SZ, P],
        "qmm_kv_plan": [P, P, I32, P, I64, P, I64, I32, P, P, P, P, I64, P, P],
        "qmm_kv_append_q4_0": [P, P, I64, P, I64, I32, P, I64, P],
        "qmm_kv_read_q4_0": [P, P, I64, P, P, P],
        "qmm_attn_q4_0": [P, P, P],
        "qmm_logits_adjust": [P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.qmm_status_string.argtypes = [ctypes.c_int]
    lib.qmm_status_string.restype = ctypes.c_char_p
    lib.qmm_version.argtypes = []
    lib.qmm_version.restype = ctypes.c_int
    for name in ("qmm_gemm_workspace_bytes", "qmm_gemm_geglu_workspace_bytes"):
        getattr(lib, name).argtypes = [I64, I64]
        getattr(lib, name).restype = SZ
    lib.qmm_attn_q4_0_workspace_bytes.argtypes = [P, I32]
    lib.qmm_attn_q4_0_workspace_bytes.restype = SZ
    lib.qmm_set_wait_timeout_ns.argtypes = [U64]
    lib.qmm_set_wait_timeout_ns.restype = None
    _lib = lib
    return lib


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


_torch = None
_raw_stream = None  # torch's own look-up of the current stream, without a Stream object


def _torch_module():
    global _torch, _raw_stream
    if _torch is None:
        import torch
        _torch = torch
        current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if current is None or device is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            _raw_stream = lambda: current(device())  # noqa: E731
    return _torch


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is None:
            _torch_module().cuda.init()
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_object(stream):
    """torch's object of a stream argument (None, the current one, stays None)."""
    cuda = _torch_module().cuda
    if stream is None or isinstance(stream, cuda.Stream):
        return stream
    return cuda.ExternalStream(_stream(stream))


def _check(status: int, where: str) -> None:
    if status != QMM_OK:
        raise QmmError(status, where)


def status_string(status: int) -> str:
    return load().qmm_status_string(int(status)).decode()


def qmm_version() -> int:
    return int(load().qmm_version())


def qmm_dequant_q4_0(w, out, n: int, k: int, stream=None) -> None:
    _check(load().qmm_dequant_q4_0(_ptr(w), _ptr(out), n, k, _stream(stream)),
           "qmm_dequant_q4_0")


def qmm_dequant_q8_0(w, out, n: int, k: int, stream=None) -> None:
    _check(load().qmm_dequant_q8_0(_ptr(w), _ptr(out), n, k, _stream(stream)),
           "qmm_dequant_q8_0")


def _ptr_pinned_ok(t) -> int:
    """Like _ptr, but a page-locked host tensor is accepted too."""
    if t is None or isinstance(t, int) or t.is_cuda:
        return _ptr(t)
    if not t.is_pinned():
        raise ValueError("host tensor must be page-locked (pin_memory())")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def qmm_copy(dst, src, nbytes: int, stream=None) -> None:
    """Stream-ordered copy by the SMs; dst and src are device memory or
    page-locked host memory."""
    _check(load().qmm_copy(_ptr_pinned_ok(dst), _ptr_pinned_ok(src), int(nbytes),
                           _stream(stream)), "qmm_copy")


def qmm_gemv_q4_0(w, x, y, m: int, n: int, k: int, stream=None) -> None:
    _check(load().qmm_gemv_q4_0(_ptr(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)),
           "qmm_gemv_q4_0")


def qmm_gemv_q8_0(w, x, y, m: int, n: int, k: int, stream=None) -> None:
    _check(load().qmm_gemv_q8_0(_ptr(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)),
           "qmm_gemv_q8_0")


def qmm_gemv_q4_0_tc(w, x, y, m: int, n: int, k: int, stream=None) -> None:
    """The Q4_0 GEMV on the tensor cores (batched decode, same accuracy bound)."""
    _check(load().qmm_gemv_q4_0_tc(_ptr(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)),
           "qmm_gemv_q4_0_tc")


def _outs(outs):
    arr = (GemvOut * max(1, len(outs)))()
    for i, (w, y, n) in enumerate(outs):
        arr[i].w = _ptr(w)
        arr[i].y = _ptr(y)
        arr[i].n = int(n)
    return arr


def qmm_gemv_q4_0_multi(outs, x, m: int, k: int, stream=None) -> None:
    """outs: sequence of (w, y, n) sharing the activations x [m][k]."""
    _check(load().qmm_gemv_q4_0_multi(_outs(outs), len(outs), _ptr(x), m, k, _stream(stream)),
           "qmm_gemv_q4_0_multi")


def qmm_gemv_q8_0_multi(outs, x, m: int, k: int, stream=None) -> None:
    _check(load().qmm_gemv_q8_0_multi(_outs(outs), len(outs), _ptr(x), m, k, _stream(stream)),
           "qmm_gemv_q8_0_multi")


def qmm_gemv_q4_0_geglu(wg, wu, x, h, m: int, n: int, k: int, stream=None) -> None:
    """h[m][n] = gelu_tanh(x . wg^T) * (x . wu^T), one launch."""
    _check(load().qmm_gemv_q4_0_geglu(_ptr(wg), _ptr(wu), _ptr(x), _ptr(h), m, n, k,
                                      _stream(stream)), "qmm_gemv_q4_0_geglu")


def qmm_gemm_q4_0(w, x_bf16, y, m: int, n: int, k: int, stream=None) -> None:
    _check(load().qmm_gemm_q4_0(_ptr(w), _ptr(x_bf16), _ptr(y), m, n, k, _stream(stream)),
           "qmm_gemm_q4_0")


def qmm_gemm_q8_0(w, x_bf16, y, m: int, n: int, k: int, stream=None) -> None:
    _check(load().qmm_gemm_q8_0(_ptr(w), _ptr(x_bf16), _ptr(y), m, n, k, _stream(stream)),
           "qmm_gemm_q8_0")


def qmm_gemm_q4_0_geglu(wg, wu, x_bf16, h_bf16, m: int, n: int, k: int, stream=None) -> None:
    """h (bf16) = gelu_tanh(X . wg^T) * (X . wu^T) on the tensor cores, one launch."""
    _check(load().qmm_gemm_q4_0_geglu(_ptr(wg), _ptr(wu), _ptr(x_bf16), _ptr(h_bf16), m, n, k,
                                      _stream(stream)), "qmm_gemm_q4_0_geglu")


def qmm_gemm_workspace_bytes(n: int, k: int, geglu: bool = False) -> int:
    lib = load()
    return int((lib.qmm_gemm_geglu_workspace_bytes if geglu else lib.qmm_gemm_workspace_bytes)(n, k))


def qmm_gemm_q4_0_ws(w, x_bf16, y, m, n, k, ws, ws_bytes, stream=None) -> None:
    _check(load().qmm_gemm_q4_0_ws(_ptr(w), _ptr(x_bf16), _ptr(y), m, n, k, _ptr(ws), int(ws_bytes),
                                   _stream(stream)), "qmm_gemm_q4_0_ws")


def qmm_gemm_q8_0_ws(w, x_bf16, y, m, n, k, ws, ws_bytes, stream=None) -> None:
    _check(load().qmm_gemm_q8_0_ws(_ptr(w), _ptr(x_bf16), _ptr(y), m, n, k, _ptr(ws), int(ws_bytes),
                                   _stream(stream)), "qmm_gemm_q8_0_ws")


def qmm_gemm_q4_0_geglu_ws(wg, wu, x_bf16, h_bf16, m, n, k, ws, ws_bytes, stream=None) -> None:
    _check(load().qmm_gemm_q4_0_geglu_ws(_ptr(wg), _ptr(wu), _ptr(x_bf16), _ptr(h_bf16), m, n, k,
                                         _ptr(ws), int(ws_bytes), _stream(stream)),
           "qmm_gemm_q4_0_geglu_ws")


def qmm_gemm_q4_0_prefill(w, x_bf16, y, m: int, n: int, k: int, stream=None) -> None:
    """The Q4_0 prefill product without a workspace argument, for callers
    that cannot allocate device memory: long prompts run in two phases on a
    64 MiB scratch array owned by the library (k <= 131072, else status
    QMM_ERR_SCRATCH).  Calls that overlap on the GPU race on that scratch."""
    _check(load().qmm_gemm_q4_0_prefill(_ptr(w), _ptr(x_bf16), _ptr(y), m, n, k, _stream(stream)),
           "qmm_gemm_q4_0_prefill")


def qmm_get_device_error(stream=None) -> int:
    """Synchronise `stream`; return (and clear) the device error word."""
    return int(load().qmm_get_device_error(_stream(stream)))


def qmm_set_wait_timeout_ns(ns: int) -> None:
    load().qmm_set_wait_timeout_ns(int(ns))


def qmm_selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(load().qmm_selftest_wait_timeout(int(timeout_ns), _stream(stream)),
           "qmm_selftest_wait_timeout")


# ---- serving operators: paged Q4_0 cache, attention, logits -------------------

class KvCacheQ4_0:
    """A paged Q4_0 cache of keys and values over the caller's four tensors:
    codes uint8 [pages][kv_heads][page_size][head_dim/2], scales float16
    [pages][kv_heads][page_size][head_dim/32].  Keeps them alive and holds
    the struct that the calls read."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        import torch
        pages, heads, page_size, half = k_codes.shape
        for codes, scales in ((k_codes, k_scales), (v_codes, v_scales)):
            if codes.dtype != torch.uint8 or scales.dtype != torch.float16:
                raise ValueError("codes must be uint8 and scales float16")
            if tuple(codes.shape) != (pages, heads, page_size, half) or \
                    tuple(scales.shape) != (pages, heads, page_size, half // 16):
                raise ValueError("codes [pages][kv_heads][page_size][head_dim/2] and scales "
                                 "[pages][kv_heads][page_size][head_dim/32] expected")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page_size, 2 * half
        self.struct = KvQ4_0(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales),
                             pages, page_size, heads, 2 * half)
        self.ref = ctypes.addressof(self.struct)


def kv_cache_q4_0(num_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda") -> KvCacheQ4_0:
    """A new cache of zeros."""
    import torch
    shape = (num_pages, kv_heads, page_size)
    codes = [torch.zeros((*shape, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros((*shape, head_dim // 32), dtype=torch.float16, device=device) for _ in range(2)]
    return KvCacheQ4_0(codes[0], scales[0], codes[1], scales[1])


def _typed(t, dtype, what: str) -> int:
    """The pointer of a contiguous tensor of this dtype (None: NULL)."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}")
    if not t.is_cuda or not t.is_contiguous():
        return _ptr(t)  # its errors
    return t.data_ptr()


def _rows(t, heads: int, dim: int, what: str):
    """(pointer, row stride, qmm_dtype) of [n][heads][dim] whose rows may lie apart."""
    dtype = t.dtype
    if dtype is _torch.float32:
        kind = QMM_F32
    elif dtype is _torch.bfloat16:
        kind = QMM_BF16
    else:
        raise ValueError(f"{what} must be float32 or bfloat16")
    n, h, d = t.shape
    row, head, one = t.stride()
    if h != heads or d != dim or (one != 1 and dim > 1) or (head != dim and heads > 1):
        raise ValueError(f"{what} must be [rows][{heads}][{dim}] with dense rows")
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    return t.data_ptr(), (row if n > 1 else heads * dim), kind


def qmm_kv_plan(cached, added, free_pages, table, page_size: int, q_start, kv_len, slots, positions, taken,
                stream=None) -> None:
    """Page tables and slot maps of the next step from the requests' lengths."""
    i32, batch, n = _torch_module().int32, cached.numel(), slots.numel()
    rows, width = table.shape
    if added.numel() != batch or rows != batch or q_start.numel() != batch + 1 or \
            kv_len.numel() != batch or positions.numel() != n:
        raise ValueError("added, table, q_start, kv_len and positions must match cached and slots in size")
    status = (_lib or load()).qmm_kv_plan(
        _typed(cached, i32, "cached"), _typed(added, i32, "added"), batch,
        _typed(free_pages, i32, "free_pages"), free_pages.numel(), _typed(table, i32, "table"),
        width, page_size, _typed(q_start, i32, "q_start"), _typed(kv_len, i32, "kv_len"),
        _typed(slots, _torch.int64, "slots"), _typed(positions, i32, "positions"), n,
        _typed(taken, i32, "taken"), _stream(stream))
    _check(status, "qmm_kv_plan")


def qmm_kv_append_q4_0(cache: KvCacheQ4_0, k, v, slots, stream=None) -> None:
    """Quantize k and v [n][kv_heads][head_dim] (fp32 or bf16) into the slots of the cache."""
    i64 = _torch_module().int64
    kp, ks, kind = _rows(k, cache.kv_heads, cache.head_dim, "k")
    vp, vs, other = _rows(v, cache.kv_heads, cache.head_dim, "v")
    n = slots.numel()
    if kind != other or k.shape[0] != n or v.shape[0] != n:
        raise ValueError("k and v must have one dtype and a row for each slot")
    status = (_lib or load()).qmm_kv_append_q4_0(cache.ref, kp, ks, vp, vs, kind, _typed(slots, i64, "slots"), n,
                                                 _stream(stream))
    _check(status, "qmm_kv_append_q4_0")


def qmm_kv_read_q4_0(cache: KvCacheQ4_0, slots, k_out, v_out, stream=None) -> None:
    """The fp32 values of cache slots, k_out and v_out [n][kv_heads][head_dim] (either may be None)."""
    f32, n = _torch_module().float32, slots.numel()
    size = n * cache.kv_heads * cache.head_dim
    if (k_out is not None and k_out.numel() != size) or (v_out is not None and v_out.numel() != size):
        raise ValueError("outputs must be [slots][kv_heads][head_dim]")
    status = (_lib or load()).qmm_kv_read_q4_0(cache.ref, _typed(slots, _torch.int64, "slots"), n,
                                               _typed(k_out, f32, "k_out"), _typed(v_out, f32, "v_out"),
                                               _stream(stream))
    _check(status, "qmm_kv_read_q4_0")


def attn_workspace(cache: KvCacheQ4_0, heads: int):
    """A workspace for attention calls on this cache (calls that overlap on the GPU need their own)."""
    import torch
    n = int(load().qmm_attn_q4_0_workspace_bytes(cache.ref, heads))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=cache.k_codes.device)


# struct qmm_attn_args and qmm_logits_args with the compiler's own padding
# (AttnArgs and LogitsArgs name the fields)
_ATTN_ARGS = struct.Struct("@PqiPqiPPqPPiqiifiiPN")
_LOGITS_ARGS = struct.Struct("@PqPqqqPPqPPPPPPPqP")


def qmm_attn_q4_0(cache: KvCacheQ4_0, q, out, table, q_start, kv_len, max_q: int, scale: float,
                  causal: bool = True, window: int = 0, lse=None, workspace=None, stream=None) -> None:
    """Attention of q [rows][heads][head_dim] (fp32 or bf16) over the cache into out (fp32 or bf16).
    Without a workspace it takes one from the memory of the stream it runs on."""
    i32 = _torch_module().int32
    rows, heads, _ = q.shape
    qp, q_stride, q_type = _rows(q, heads, cache.head_dim, "q")
    op, out_stride, out_type = _rows(out, heads, cache.head_dim, "out")
    batch = kv_len.numel()
    tables, width = table.shape
    if out.shape[0] != rows or tables != batch or q_start.numel() != batch + 1 or \
            (lse is not None and lse.numel() != rows * heads):
        raise ValueError("out, lse, table and q_start must match q and kv_len in size")
    if workspace is None:
        # the tensor dies with this call: its bytes go back to the pool of the
        # stream it was taken under, which must be the one that uses them
        with _torch.cuda.stream(_stream_object(stream)):
            workspace = attn_workspace(cache, heads)
    args = _ATTN_ARGS.pack(qp, q_stride, q_type, op, out_stride, out_type, _typed(lse, _torch.float32, "lse"),
                           _typed(table, i32, "table"), width, _typed(q_start, i32, "q_start"),
                           _typed(kv_len, i32, "kv_len"), batch, rows, max_q, heads, scale, bool(causal), window,
                           _ptr(workspace), workspace.numel() * workspace.element_size())
    _check((_lib or load()).qmm_attn_q4_0(cache.ref, args, _stream(stream)), "qmm_attn_q4_0")


def qmm_logits_adjust(logits, out, history=None, hist_start=None, prompt_len=None, repetition=None,
                      frequency=None, presence=None, bias_ids=None, bias_values=None, bias_start=None,
                      allowed=None, stream=None) -> None:
    """Penalties, biases and grammar masks on logits [rows][vocab] (fp32); out may be logits."""
    torch = _torch_module()
    i32, f32 = torch.int32, torch.float32
    rows, vocab = logits.shape
    for t in (logits, out):
        if t.dtype is not f32 or t.shape != logits.shape or (t.stride(1) != 1 and vocab > 1) or not t.is_cuda:
            raise ValueError("logits and out must be float32 [rows][vocab] on a CUDA device with dense rows")
    for t, n, what in ((hist_start, rows + 1, "hist_start"), (bias_start, rows + 1, "bias_start"),
                       (prompt_len, rows, "prompt_len"), (repetition, rows, "repetition"),
                       (frequency, rows, "frequency"), (presence, rows, "presence"),
                       (allowed, rows * ((vocab + 31) // 32), "allowed")):
        if t is not None and t.numel() != n:
            raise ValueError(f"{what} must have {n} entries")
    if (bias_ids is None) != (bias_values is None) or \
            (bias_ids is not None and bias_ids.numel() != bias_values.numel()):
        raise ValueError("bias_ids and bias_values go together")
    args = _LOGITS_ARGS.pack(
        logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, out.data_ptr(),
        out.stride(0) if rows > 1 else vocab, rows, vocab, _typed(history, i32, "history"),
        _typed(hist_start, i32, "hist_start"), 0 if history is None else history.numel(),
        _typed(prompt_len, i32, "prompt_len"), _typed(repetition, f32, "repetition"),
        _typed(frequency, f32, "frequency"), _typed(presence, f32, "presence"), _typed(bias_ids, i32, "bias_ids"),
        _typed(bias_values, f32, "bias_values"), _typed(bias_start, i32, "bias_start"),
        0 if bias_ids is None else bias_ids.numel(), _typed(allowed, i32, "allowed"))
    _check((_lib or load()).qmm_logits_adjust(args, _stream(stream)), "qmm_logits_adjust")


# ---- tensor-level conveniences (allocate the output, then call the ABI) ----

def dequant(fmt: str, w, n: int, k: int, stream=None):
    import torch
    out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    (qmm_dequant_q4_0 if fmt == "q4_0" else qmm_dequant_q8_0)(w, out, n, k, stream)
    return out


def gemv(fmt: str, w, x, n: int, k: int, stream=None):
    import torch
    m = x.shape[0]
    y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    (qmm_gemv_q4_0 if fmt == "q4_0" else qmm_gemv_q8_0)(w, x, y, m, n, k, stream)
    return y


def gemv_tc_q4_0(w, x, n: int, k: int, stream=None):
    import torch
    m = x.shape[0]
    y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    qmm_gemv_q4_0_tc(w, x, y, m, n, k, stream)
    return y


def geglu_q4_0(wg, wu, x, n: int, k: int, stream=None):
    import torch
    m = x.shape[0]
    h = torch.empty((m, n), dtype=torch.float32, device=x.device)
    qmm_gemv_q4_0_geglu(wg, wu, x, h, m, n, k, stream)
    return h


def gemm(fmt: str, w, x_bf16, n: int, k: int, stream=None, workspace=None):
    """workspace: a device tensor of at least qmm_gemm_workspace_bytes(n, k) bytes
    (the two-phase path for m > 256), or None (the fused call)."""
    import torch
    m = x_bf16.shape[0]
    y = torch.empty((m, n), dtype=torch.float32, device=x_bf16.device)
    if workspace is None:
        (qmm_gemm_q4_0 if fmt == "q4_0" else qmm_gemm_q8_0)(w, x_bf16, y, m, n, k, stream)
    else:
        (qmm_gemm_q4_0_ws if fmt == "q4_0" else qmm_gemm_q8_0_ws)(
            w, x_bf16, y, m, n, k, workspace, workspace.numel() * workspace.element_size(), stream)
    return y


def gemm_geglu_q4_0(wg, wu, x_bf16, n: int, k: int, stream=None, workspace=None):
    """Returns h as an int16 tensor of bf16 bit patterns [m][n]."""
    import torch
    m = x_bf16.shape[0]
    h = torch.empty((m, n), dtype=torch.int16, device=x_bf16.device)
    if workspace is None:
        qmm_gemm_q4_0_geglu(wg, wu, x_bf16, h, m, n, k, stream)
    else:
        qmm_gemm_q4_0_geglu_ws(wg, wu, x_bf16, h, m, n, k, workspace,
                               workspace.numel() * workspace.element_size(), stream)
    return h


def gemm_q4_0(w, x_bf16, n: int, k: int, stream=None):
    import torch
    m = x_bf16.shape[0]
    y = torch.empty((m, n), dtype=torch.float32, device=x_bf16.device)
    qmm_gemm_q4_0(w, x_bf16, y, m, n, k, stream)
    return y
