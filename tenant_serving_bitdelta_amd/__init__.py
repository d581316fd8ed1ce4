"""Python binding of libbitdelta (the MI355X BitDelta hot path).

Thin ctypes marshalling only: every step of compression and of the fused reconstruct-and-
multiply runs in the library's HIP kernels.  torch is used to hold device memory and to name
the current HIP stream.  If the library is not built this module raises on first use; there
is no fallback of any kind.

Every call runs on ``stream``, a raw HIP stream handle (None: torch's current stream).  What it
allocates itself is allocated on that stream; a call waits for no other stream's work, nor does
any other stream wait for it.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

__all__ = [
    "BitDeltaError", "lib", "abi_version", "sign_words", "compress_workspace_bytes",
    "compress_rows", "compress_rows_workspace_bytes", "compress_from_weights",
    "compress", "plan_segments", "matmul", "matmul_grouped", "auto_path", "PATHS",
    "matmul_workspace_bytes", "sign_words_t128", "reconstruct", "upload_variant", "Residency",
    "matmul_grouped_noalloc", "NOALLOC_SCRATCH_BYTES", "attend_shared",
    "attend_shared_workspace_bytes", "attend_window", "attend_window_workspace_bytes", "sample",
    "cache_write", "cache_read",
]

ABI_VERSION = 7
NOALLOC_SCRATCH_BYTES = 128 << 20  # BITDELTA_NOALLOC_SCRATCH_BYTES

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbitdelta.so")

PATHS = {"auto": 0, "gemv": 1, "stream": 2, "prefill": 3, "split": 4}
_OUT = {"bf16": 0, "f32": 1}
MAX_VARIANTS = 64
MAX_PROBLEMS = 8


class BitDeltaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        name = _lib().bitdelta_status_string(int(status)).decode() if _LIB is not None else str(status)
        if self.status == 6 and _LIB is not None:  # BITDELTA_ERR_HIP: name the runtime's error
            name += f" [{_LIB.bitdelta_last_hip_error_string().decode()}]"
        super().__init__(f"{what}: {name} (status {status})" if what else f"{name} (status {status})")


class _Variant(ctypes.Structure):
    _fields_ = [("sign_words", ctypes.c_void_p), ("sign_words_t128", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("alpha_per_row", ctypes.c_int32)]


class _Problem(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("w_base", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("d_out", ctypes.c_int64), ("d_in", ctypes.c_int64),
        ("variants", ctypes.POINTER(_Variant)), ("num_variants", ctypes.c_int32),
    ]


class _KvCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("k_stride_page", ctypes.c_int64), ("k_stride_token", ctypes.c_int64),
        ("k_stride_head", ctypes.c_int64), ("v_stride_page", ctypes.c_int64),
        ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("k_block_scales", ctypes.c_void_p), ("v_block_scales", ctypes.c_void_p),
    ]


class _KvRows(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("tokens", ctypes.c_int64),
        ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
    ]


class _AttendRows(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("tokens", ctypes.c_int64), ("heads", ctypes.c_int32),
        ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
        ("scale", ctypes.c_float),
    ]


_LIB = None
_i32p = ctypes.POINTER(ctypes.c_int32)


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950) first")
        # torch first: its HIP runtime is then the one the library binds to.  Loaded the other
        # way round, a process can end up with two HIP runtimes (torch's bundled copy and the
        # system one) whose kernels and device memory do not mix.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        # entry points that came without a new ABI version
        for name in ("bitdelta_attend_shared", "bitdelta_attend_window", "bitdelta_sample",
                     "bitdelta_cache_write", "bitdelta_cache_read"):
            if not hasattr(L, name):
                raise RuntimeError(f"{LIB_PATH} has no {name}: it is older than this package; run "
                                   "__graft_entry__.build() again")
        L.bitdelta_abi_version.restype = ctypes.c_int
        L.bitdelta_status_string.restype = ctypes.c_char_p
        L.bitdelta_status_string.argtypes = [ctypes.c_int]
        L.bitdelta_last_hip_error.restype = ctypes.c_int32
        L.bitdelta_last_hip_error_string.restype = ctypes.c_char_p
        L.bitdelta_sign_words.restype = ctypes.c_int64
        L.bitdelta_sign_words.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.bitdelta_compress_workspace_bytes.restype = ctypes.c_size_t
        L.bitdelta_compress_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.bitdelta_compress.restype = ctypes.c_int
        L.bitdelta_compress.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_compress_from_weights.restype = ctypes.c_int
        L.bitdelta_compress_from_weights.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                     ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_compress_rows.restype = ctypes.c_int
        L.bitdelta_compress_rows.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_compress_rows_workspace_bytes.restype = ctypes.c_size_t
        L.bitdelta_compress_rows_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.bitdelta_residency_create.restype = ctypes.c_int
        L.bitdelta_residency_create.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64),
                                                ctypes.c_int64, ctypes.c_int32,
                                                ctypes.POINTER(ctypes.c_void_p)]
        L.bitdelta_residency_destroy.restype = None
        L.bitdelta_residency_destroy.argtypes = [ctypes.c_void_p]
        L.bitdelta_residency_request.restype = ctypes.c_int
        L.bitdelta_residency_request.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                                 _i32p, _i32p, _i32p]
        L.bitdelta_residency_release.restype = ctypes.c_int
        L.bitdelta_residency_release.argtypes = [ctypes.c_void_p, ctypes.c_int32]
        L.bitdelta_residency_holds.restype = ctypes.c_int64
        L.bitdelta_residency_holds.argtypes = [ctypes.c_void_p, ctypes.c_int32]
        L.bitdelta_residency_load_enqueued.restype = ctypes.c_int
        L.bitdelta_residency_load_enqueued.argtypes = [ctypes.c_void_p, ctypes.c_int32,
                                                       ctypes.c_void_p]
        L.bitdelta_residency_poll.restype = ctypes.c_int
        L.bitdelta_residency_poll.argtypes = [ctypes.c_void_p, _i32p, _i32p]
        L.bitdelta_reconstruct.restype = ctypes.c_int
        L.bitdelta_reconstruct.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.POINTER(_Variant), ctypes.c_void_p,
                                           ctypes.c_void_p]
        L.bitdelta_upload_variant.restype = ctypes.c_int
        L.bitdelta_upload_variant.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                              ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_residency_load_done.restype = ctypes.c_int
        L.bitdelta_residency_load_done.argtypes = [ctypes.c_void_p, ctypes.c_int32]
        L.bitdelta_residency_state.restype = ctypes.c_int32
        L.bitdelta_residency_state.argtypes = [ctypes.c_void_p, ctypes.c_int32]
        L.bitdelta_residency_used_bytes.restype = ctypes.c_int64
        L.bitdelta_residency_used_bytes.argtypes = [ctypes.c_void_p]
        L.bitdelta_sign_words_t128.restype = ctypes.c_int64
        L.bitdelta_sign_words_t128.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.bitdelta_plan_segments.restype = ctypes.c_int
        L.bitdelta_plan_segments.argtypes = [_i32p, ctypes.c_int64, ctypes.c_int32, _i32p, _i32p,
                                             _i32p, _i32p]
        L.bitdelta_matmul.restype = ctypes.c_int
        L.bitdelta_matmul.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_Variant),
                                      ctypes.c_int32, _i32p, _i32p, ctypes.c_int32,
                                      ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                      ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_matmul_grouped.restype = ctypes.c_int
        L.bitdelta_matmul_grouped.argtypes = [ctypes.POINTER(_Problem), ctypes.c_int32,
                                              ctypes.c_int64, _i32p, _i32p, ctypes.c_int32,
                                              ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                              ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_matmul_grouped_noalloc.restype = ctypes.c_int
        L.bitdelta_matmul_grouped_noalloc.argtypes = [ctypes.POINTER(_Problem), ctypes.c_int32,
                                                      ctypes.c_int64, _i32p, _i32p, ctypes.c_int32,
                                                      ctypes.c_int32, ctypes.c_int32,
                                                      ctypes.c_void_p]
        L.bitdelta_matmul_workspace_bytes.restype = ctypes.c_size_t
        L.bitdelta_matmul_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64,
                                                      ctypes.c_int32]
        L.bitdelta_auto_path.restype = ctypes.c_int32
        L.bitdelta_auto_path.argtypes = [ctypes.c_int64, _i32p, _i32p, ctypes.c_int32]
        rows_p, cache_p = ctypes.POINTER(_AttendRows), ctypes.POINTER(_KvCache)
        L.bitdelta_attend_shared.restype = ctypes.c_int
        L.bitdelta_attend_shared.argtypes = [rows_p, cache_p, ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_attend_shared_workspace_bytes.restype = ctypes.c_size_t
        L.bitdelta_attend_shared_workspace_bytes.argtypes = [
            ctypes.c_int64, ctypes.c_int32, cache_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
            ctypes.c_int32]
        L.bitdelta_attend_window.restype = ctypes.c_int
        L.bitdelta_attend_window.argtypes = [rows_p, cache_p, ctypes.c_int32, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.bitdelta_attend_window_workspace_bytes.restype = ctypes.c_size_t
        L.bitdelta_attend_window_workspace_bytes.argtypes = [
            ctypes.c_int64, ctypes.c_int32, cache_p, ctypes.c_int32, ctypes.c_int32,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
        for f in (L.bitdelta_cache_write, L.bitdelta_cache_read):
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.POINTER(_KvRows), cache_p, ctypes.c_int32, ctypes.c_void_p,
                          ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.bitdelta_sample.restype = ctypes.c_int
        L.bitdelta_sample.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int64, *[ctypes.c_void_p] * 8]
        _LIB = L
    return _LIB


lib = _lib


def _check(status: int, what: str):
    if status != 0:
        raise BitDeltaError(status, what)


def _i32(a):
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return arr, arr.ctypes.data_as(_i32p)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _raw_stream(stream, tensor):
    """The call's stream handle: ``stream``, or torch's current one on the tensor's device (in 0.1 us;
    through torch.cuda.current_stream and its object it takes 1.9 of a short call's 10)."""
    if stream is not None:
        return int(stream)
    import torch
    return torch._C._cuda_getCurrentRawStream(tensor.device.index)


def _empty(shape, dtype, device, stream, kept=True):
    """An uninitialised device tensor for a call whose kernels run on ``stream`` (None: torch's
    current stream).  torch's caching allocator orders a block's uses by the stream it was allocated
    on: a block freed on the current stream may still be in use by that stream's queued work, which
    ``stream`` does not wait for.  So on another stream the tensor is allocated there, and, if the
    caller gets it (``kept``), recorded as in use on the current one.  (Calls of some 10 us make their
    results themselves where ``stream`` is None: through here one takes 2 us longer.)"""
    import torch
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if int(stream) == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    if kept:
        t.record_stream(current)
    return t


def _temp(nbytes, device, stream, dtype_name="uint8"):
    """A scratch device tensor for one call whose kernels run on ``stream`` (None: torch's
    current stream)."""
    import torch
    dtype = getattr(torch, dtype_name)
    n = max(int(nbytes), 1) // dtype.itemsize
    return _empty(max(n, 1), dtype, device, stream, kept=False)


def _numel_at_least(t, n, what):
    if t.numel() < n:
        raise ValueError(f"{what} holds {t.numel()} elements, needs at least {n}")


def _numel_exact(t, n, what):
    if t.numel() != n:
        raise ValueError(f"{what} holds {t.numel()} elements, needs exactly {n}")


def _check_shape(t, shape, what):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, needs {tuple(shape)}")


_DTYPES = {}


def _dev(t, dtype_name, what):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA/HIP torch tensor")
    want = _DTYPES.get(dtype_name)
    if want is None:
        want = _DTYPES[dtype_name] = getattr(torch, dtype_name.split(".")[1])
    if t.dtype is not want:
        raise TypeError(f"{what} must be {dtype_name}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def abi_version() -> int:
    return int(_lib().bitdelta_abi_version())


def sign_words(d_out: int, d_in: int) -> int:
    return int(_lib().bitdelta_sign_words(d_out, d_in))


def sign_words_t128(d_out: int, d_in: int) -> int:
    """Words of the tiled sign copy (128-row blocks x 128-column steps), -1 if d_in % 128."""
    return int(_lib().bitdelta_sign_words_t128(d_out, d_in))


def compress_workspace_bytes(d_out: int, d_in: int) -> int:
    return int(_lib().bitdelta_compress_workspace_bytes(d_out, d_in))


def _compress_outputs(d_out, d_in, words, tiled, alpha, alpha_n):
    """Pointers of compress outputs after checking their sizes: ``words`` (int32, d_out * d_in / 32
    elements) and ``tiled`` (int32, at least sign_words_t128 elements) may each be None, not both."""
    if words is None and tiled is None:
        raise ValueError("give the row-major words, the tiled words, or both")
    if d_in % 32:
        raise ValueError("d_in must be a multiple of 32")
    wptr = tptr = None
    if words is not None:
        _numel_exact(words, d_out * d_in // 32, "words")
        wptr = _dev(words, "torch.int32", "words")
    if tiled is not None:
        nt = sign_words_t128(d_out, d_in)
        if nt < 0:
            raise ValueError("the tiled layout needs d_in % 128 == 0")
        _numel_at_least(tiled, nt, "tiled sign words")
        tptr = _dev(tiled, "torch.int32", "tiled sign words")
    _numel_exact(alpha, alpha_n, "alpha")
    return wptr, tptr, _dev(alpha, "torch.float32", "alpha")


def _workspace_arg(workspace, need, device, stream):
    """(tensor, pointer, bytes) of a caller's workspace (the library checks its size), or of a
    scratch tensor sized ``need`` when None."""
    if workspace is None:
        workspace = _temp(max(need, 8), device, stream, "float64")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def compress(delta, words, alpha, workspace=None, stream=None, tiled=None):
    """alpha = mean|delta| and packed sign bits of one float32 [d_out, d_in] matrix.
    ``words``: int32 tensor [d_out, d_in // 32] (uint32 bit patterns) or None, ``alpha``: float32
    [1], ``tiled``: int32 tensor of sign_words_t128(d_out, d_in) words for the tiled layout, or
    None (at least one of words / tiled)."""
    d_out, d_in = delta.shape
    wptr, tptr, aptr = _compress_outputs(d_out, d_in, words, tiled, alpha, 1)
    ws, ws_ptr, ws_bytes = _workspace_arg(workspace, compress_workspace_bytes(d_out, d_in),
                                          delta.device, stream)
    _check(_lib().bitdelta_compress(
        _dev(delta, "torch.float32", "delta"), d_out, d_in, wptr, tptr, aptr, ws_ptr, ws_bytes,
        _stream(stream)), "bitdelta_compress")
    return words, alpha


def compress_from_weights(w_ft, w_base, words, alpha, workspace=None, stream=None, tiled=None):
    """compress() of Delta = w_ft - w_base for two bf16 [d_out, d_in] matrices, Delta never
    formed.  Outputs as for compress()."""
    d_out, d_in = w_base.shape
    if tuple(w_ft.shape) != (d_out, d_in):
        raise ValueError("w_ft and w_base must have the same shape")
    wptr, tptr, aptr = _compress_outputs(d_out, d_in, words, tiled, alpha, 1)
    ws, ws_ptr, ws_bytes = _workspace_arg(workspace, compress_workspace_bytes(d_out, d_in),
                                          w_base.device, stream)
    _check(_lib().bitdelta_compress_from_weights(
        _dev(w_ft, "torch.bfloat16", "w_ft"), _dev(w_base, "torch.bfloat16", "w_base"), d_out, d_in,
        wptr, tptr, aptr, ws_ptr, ws_bytes, _stream(stream)), "bitdelta_compress_from_weights")
    return words, alpha


def compress_rows_workspace_bytes(d_out: int, d_in: int) -> int:
    return int(_lib().bitdelta_compress_rows_workspace_bytes(d_out, d_in))


def compress_rows(delta, words, alpha, workspace=None, stream=None, tiled=None):
    """compress() with one scale per output row: ``alpha`` is float32 [d_out]; pass the result to
    matmul as (words, alpha[, tiled]) and it is applied row by row."""
    d_out, d_in = delta.shape
    wptr, tptr, aptr = _compress_outputs(d_out, d_in, words, tiled, alpha, d_out)
    ws, ws_ptr, ws_bytes = _workspace_arg(workspace, compress_rows_workspace_bytes(d_out, d_in),
                                          delta.device, stream)
    _check(_lib().bitdelta_compress_rows(
        _dev(delta, "torch.float32", "delta"), d_out, d_in, wptr, tptr, aptr, ws_ptr, ws_bytes,
        _stream(stream)), "bitdelta_compress_rows")
    return words, alpha


def plan_segments(token_variant, num_variants: int):
    """Stable grouping of tokens by variant (base -1 first).  Returns numpy int32
    (perm, seg_offsets, seg_variant)."""
    ids, ids_p = _i32(token_variant)
    m = ids.size
    perm = np.zeros(max(m, 1), dtype=np.int32)
    offs = np.zeros(num_variants + 2, dtype=np.int32)
    segv = np.zeros(num_variants + 1, dtype=np.int32)
    ns = ctypes.c_int32(0)
    _check(_lib().bitdelta_plan_segments(
        ids_p, m, num_variants, perm.ctypes.data_as(_i32p), offs.ctypes.data_as(_i32p),
        segv.ctypes.data_as(_i32p), ctypes.byref(ns)), "bitdelta_plan_segments")
    n = ns.value
    return perm[:m].copy(), offs[:n + 1].copy(), segv[:n].copy()


def matmul_workspace_bytes(m: int, d_in: int, path="auto") -> int:
    """Device workspace one linear of a matmul call on ``path`` needs (bytes, 0 if none)."""
    return int(_lib().bitdelta_matmul_workspace_bytes(m, d_in, PATHS[path]))


def _workspace(workspace, need, device, stream):
    """(pointer, bytes, tensor) of the caller's workspace tensor, or of a scratch one sized
    ``need`` when None (none at all when ``need`` is 0)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _temp(need, device, stream)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def auto_path(m: int, seg_offsets, seg_variant) -> int:
    o, op = _i32(seg_offsets)
    v, vp = _i32(seg_variant)
    return int(_lib().bitdelta_auto_path(m, op, vp, v.size))


def _variant_struct(v, item, d_out, d_in, i=0):
    """Fill one _Variant from (words, alpha) or (words, alpha, tiled_words): words (row-major,
    d_out * d_in / 32 int32) or tiled_words (at least sign_words_t128 int32) may be None, not both;
    alpha holds one float32 (per matrix) or d_out of them (per output row)."""
    words, alpha = item[0], item[1]
    tiled = item[2] if len(item) > 2 else None
    if words is None and tiled is None:
        raise ValueError(f"variant {i}: needs row-major or tiled sign words")
    if words is not None:
        _numel_exact(words, d_out * d_in // 32, f"variant {i} sign words")
        v.sign_words = _dev(words, "torch.int32", "sign words")
    if tiled is not None:
        nt = sign_words_t128(d_out, d_in)
        if nt < 0:
            raise ValueError(f"variant {i}: tiled sign words need d_in % 128 == 0")
        _numel_at_least(tiled, nt, f"variant {i} tiled sign words")
        v.sign_words_t128 = _dev(tiled, "torch.int32", "tiled sign words")
    n = alpha.numel()
    if n != 1 and n != d_out:
        raise ValueError(f"variant {i}: alpha must hold 1 or d_out = {d_out} values, not {n}")
    v.alpha = _dev(alpha, "torch.float32", "alpha")
    v.alpha_per_row = 1 if n > 1 else 0


def _variants_array(variants, d_out, d_in):
    """variants: list of (words, alpha[, tiled_words]) tuples (None for ids the call never uses)."""
    arr = (_Variant * max(len(variants), 1))()
    for i, item in enumerate(variants):
        if item is not None:
            _variant_struct(arr[i], item, d_out, d_in, i)
    return arr


def _problems_array(problems, m, out_dtype):
    """ctypes array of bitdelta_problem for (x, w_base, y, variants) tuples, sizes checked; the
    second value keeps the variant arrays alive."""
    if not 1 <= len(problems) <= MAX_PROBLEMS:
        raise ValueError("1..8 problems per call")
    parr = (_Problem * len(problems))()
    keep = []
    for i, (x, w, y, variants) in enumerate(problems):
        if w.dim() != 2:
            raise ValueError("w_base must be [d_out, d_in]")
        d_out, d_in = int(w.shape[0]), int(w.shape[1])
        _check_shape(x, (m, d_in), f"problem {i} x")
        _check_shape(y, (m, d_out), f"problem {i} y")
        varr = _variants_array(variants, d_out, d_in)
        keep.append(varr)
        parr[i].x = _dev(x, "torch.bfloat16", "x")
        parr[i].w_base = _dev(w, "torch.bfloat16", "w_base")
        parr[i].y = _dev(y, "torch.bfloat16" if out_dtype == "bf16" else "torch.float32", "y")
        parr[i].d_out, parr[i].d_in = d_out, d_in
        parr[i].variants = ctypes.cast(varr, ctypes.POINTER(_Variant))
        parr[i].num_variants = len(variants)
    return parr, keep


def matmul_grouped(problems, seg_offsets, seg_variant, out_dtype="bf16", path="auto", stream=None,
                   workspace=None):
    """Fused y = x (W_base + alpha_v sign_v)^T for several linears sharing one segmentation.
    ``problems``: list of (x, w_base, y, variants) with variants a list of (words, alpha).
    ``workspace``: device tensor of at least the summed matmul_workspace_bytes (allocated here
    when None)."""
    offs, offs_p = _i32(seg_offsets)
    segv, segv_p = _i32(seg_variant)
    m = int(offs[-1]) if offs.size else 0
    parr, keep = _problems_array(problems, m, out_dtype)
    # the library checks the size of a caller's workspace itself; only a missing one is sized here
    need = 0 if workspace is not None else sum(
        matmul_workspace_bytes(m, int(w.shape[1]), path) for _, w, _, _ in problems)
    ws_ptr, ws_bytes, ws = _workspace(workspace, need, problems[0][1].device, stream)
    _check(_lib().bitdelta_matmul_grouped(parr, len(problems), m, offs_p, segv_p, segv.size,
                                          _OUT[out_dtype], PATHS[path], ws_ptr, ws_bytes,
                                          _stream(stream)),
           "bitdelta_matmul_grouped")
    return [p[2] for p in problems]


def matmul_grouped_noalloc(problems, seg_offsets, seg_variant, out_dtype="bf16", path="auto",
                           stream=None):
    """matmul_grouped on the SPLIT path with the library's own per-device scratch as workspace:
    the call allocates no device memory (for callers that cannot).  Batches the SPLIT path does
    not serve raise BitDeltaError (status 5); calls that overlap on one device must not be made."""
    offs, offs_p = _i32(seg_offsets)
    segv, segv_p = _i32(seg_variant)
    m = int(offs[-1]) if offs.size else 0
    parr, keep = _problems_array(problems, m, out_dtype)
    _check(_lib().bitdelta_matmul_grouped_noalloc(parr, len(problems), m, offs_p, segv_p, segv.size,
                                                  _OUT[out_dtype], PATHS[path], _stream(stream)),
           "bitdelta_matmul_grouped_noalloc")
    return [p[2] for p in problems]


def matmul(x, w_base, variants, seg_offsets, seg_variant, y=None, out_dtype="bf16", path="auto",
           stream=None, workspace=None):
    """Fused y = x (W_base + alpha_v sign_v)^T over a token batch grouped by variant."""
    import torch
    if y is None:
        y = _empty((x.shape[0], w_base.shape[0]),
                   torch.bfloat16 if out_dtype == "bf16" else torch.float32, x.device, stream)
    if path != "auto":
        matmul_grouped([(x, w_base, y, variants)], seg_offsets, seg_variant, out_dtype, path,
                       stream, workspace)
        return y
    offs, offs_p = _i32(seg_offsets)
    segv, segv_p = _i32(seg_variant)
    if w_base.dim() != 2:
        raise ValueError("w_base must be [d_out, d_in]")
    d_out, d_in = int(w_base.shape[0]), int(w_base.shape[1])
    m = int(offs[-1]) if offs.size else 0
    _check_shape(x, (m, d_in), "x")
    _check_shape(y, (m, d_out), "y")
    varr = _variants_array(variants, d_out, d_in)
    ws_ptr, ws_bytes, ws = _workspace(
        workspace, 0 if workspace is not None else matmul_workspace_bytes(m, d_in), x.device, stream)
    _check(_lib().bitdelta_matmul(
        _dev(x, "torch.bfloat16", "x"), _dev(w_base, "torch.bfloat16", "w_base"),
        m, d_out, d_in, varr, len(variants),
        offs_p, segv_p, segv.size,
        _dev(y, "torch.bfloat16" if out_dtype == "bf16" else "torch.float32", "y"),
        _OUT[out_dtype], ws_ptr, ws_bytes, _stream(stream)), "bitdelta_matmul")
    return y


class Residency:
    """The library's delta residency manager (host only): request(v) -> (action, evicted ids),
    with action one of HIT, LOAD, QUEUED, NO_ROOM; load_done(v) when a load has finished."""
    HIT, LOAD, QUEUED, NO_ROOM = 0, 1, 2, 3
    ABSENT, LOADING, RESIDENT = 0, 1, 2

    def __init__(self, variant_bytes, capacity_bytes: int, num_pinned: int = 6):
        L = _lib()
        self._n = len(variant_bytes)
        sizes = (ctypes.c_int64 * max(self._n, 1))(*[int(b) for b in variant_bytes])
        h = ctypes.c_void_p()
        _check(L.bitdelta_residency_create(self._n, sizes, int(capacity_bytes), int(num_pinned),
                                           ctypes.byref(h)), "bitdelta_residency_create")
        self._h = h

    def request(self, v: int, hold: bool = False):
        """(action, evicted ids).  hold=True: an answer other than NO_ROOM makes this request a
        holder of v, which is not evicted until release(v)."""
        # output buffers per call, so that threads sharing a manager never read each other's
        ev = (ctypes.c_int32 * self._n)()
        act, ne = ctypes.c_int32(), ctypes.c_int32()
        _check(_lib().bitdelta_residency_request(self._h, int(v), 1 if hold else 0,
                                                 ctypes.byref(act), ev, ctypes.byref(ne)),
               "bitdelta_residency_request")
        return act.value, [ev[i] for i in range(ne.value)]

    def release(self, v: int):
        _check(_lib().bitdelta_residency_release(self._h, int(v)), "bitdelta_residency_release")

    def holds(self, v: int) -> int:
        return int(_lib().bitdelta_residency_holds(self._h, int(v)))

    def load_enqueued(self, v: int, event):
        """Attach the event recorded after v's upload (a torch.cuda.Event that has been
        recorded); poll() then makes v resident once the event has completed.  Keep the event
        alive until then."""
        _check(_lib().bitdelta_residency_load_enqueued(self._h, int(v),
                                                       ctypes.c_void_p(int(event.cuda_event))),
               "bitdelta_residency_load_enqueued")

    def poll(self):
        """Variants whose attached upload event has completed since the last poll (now resident)."""
        out = (ctypes.c_int32 * self._n)()
        nc = ctypes.c_int32()
        _check(_lib().bitdelta_residency_poll(self._h, out, ctypes.byref(nc)),
               "bitdelta_residency_poll")
        return [out[i] for i in range(nc.value)]

    def load_done(self, v: int):
        _check(_lib().bitdelta_residency_load_done(self._h, int(v)), "bitdelta_residency_load_done")

    def state(self, v: int) -> int:
        return int(_lib().bitdelta_residency_state(self._h, int(v)))

    def used_bytes(self) -> int:
        return int(_lib().bitdelta_residency_used_bytes(self._h))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _LIB is not None:
            _LIB.bitdelta_residency_destroy(h)
            self._h = None


def reconstruct(w_base, variant, w_eff=None, stream=None):
    """W_eff = bf16(W_base + alpha * sign) written to a bf16 [d_out, d_in] tensor (the unfused
    reconstruction; the fused matmul never forms it).  ``variant``: (words, alpha[, tiled])."""
    import torch
    if w_base.dim() != 2:
        raise ValueError("w_base must be [d_out, d_in]")
    d_out, d_in = int(w_base.shape[0]), int(w_base.shape[1])
    if w_eff is None:
        w_eff = _empty((d_out, d_in), torch.bfloat16, w_base.device, stream)
    _check_shape(w_eff, (d_out, d_in), "w_eff")
    v = _Variant()
    _variant_struct(v, variant, d_out, d_in)
    _check(_lib().bitdelta_reconstruct(_dev(w_base, "torch.bfloat16", "w_base"), d_out, d_in,
                                       ctypes.byref(v), _dev(w_eff, "torch.bfloat16", "w_eff"),
                                       _stream(stream)), "bitdelta_reconstruct")
    return w_eff


def upload_variant(host_words, host_alpha, d_out: int, d_in: int, words=None, tiled=None,
                   alpha=None, staging=None, stream=None):
    """Host -> device upload of one compressed matrix of a variant, into the layout the kernels
    read.  ``host_words``: CPU int32 tensor of d_out * d_in / 32 row-major words (pinned memory
    makes the copy asynchronous); ``host_alpha``: CPU float32 tensor of 1 or d_out scales;
    ``words`` / ``tiled``: device destinations (at least one); ``alpha``: device float32
    destination; ``staging``: device scratch of d_out * d_in / 8 bytes when only ``tiled`` is
    given (allocated here when None).  Returns (words, tiled, alpha)."""
    import torch
    if host_words.is_cuda or host_alpha.is_cuda:
        raise TypeError("host_words and host_alpha must be CPU tensors")
    if host_words.dtype is not torch.int32 or host_alpha.dtype is not torch.float32:
        raise TypeError("host_words must be int32 and host_alpha float32")
    if not host_words.is_contiguous() or not host_alpha.is_contiguous():
        raise ValueError("host tensors must be contiguous")
    if d_in % 32:
        raise ValueError("d_in must be a multiple of 32")
    _numel_exact(host_words, d_out * d_in // 32, "host_words")
    na = host_alpha.numel()
    if na != 1 and na != d_out:
        raise ValueError("host_alpha must hold 1 or d_out scales")
    if alpha is None:
        raise ValueError("a device alpha tensor is required")
    wptr, tptr, aptr = _compress_outputs(d_out, d_in, words, tiled, alpha, na)
    sptr, sbytes = None, 0
    if words is None:
        nb = d_out * d_in // 8
        if staging is None:
            staging = _temp(nb, alpha.device, stream)
        if not staging.is_cuda or not staging.is_contiguous():
            raise ValueError("staging must be a contiguous device tensor")
        sptr, sbytes = staging.data_ptr(), staging.numel() * staging.element_size()
    _check(_lib().bitdelta_upload_variant(host_words.data_ptr(), host_alpha.data_ptr(), na, d_out,
                                          d_in, wptr, tptr, aptr, sptr, sbytes, _stream(stream)),
           "bitdelta_upload_variant")
    return words, tiled, alpha


# ---------------------------------------------------------------------------------------------
# Attention over a paged cache
# ---------------------------------------------------------------------------------------------

_KV_DTYPES = {}  # torch dtype -> bitdelta_kv_dtype


def _block_scales(pages, scales, what):
    """Address of a 4-bit cache's scale bytes: [pages, page_size, kv_heads, head_dim / 32] laid out as
    the pages are, at a 16th of their byte offsets."""
    import torch
    if not isinstance(scales, torch.Tensor) or not scales.is_cuda:
        raise TypeError(f"{what}_block_scales must be a CUDA/HIP torch tensor (4-bit pages have them)")
    if scales.dtype is not torch.uint8:
        raise TypeError(f"{what}_block_scales must be torch.uint8, got {scales.dtype}")
    if scales.device != pages.device:
        raise ValueError(f"{what}_block_scales are on {scales.device}, the pages on {pages.device}")
    shape = pages.shape
    if scales.shape != (shape[0], shape[1], shape[2], shape[3] // 16):
        raise ValueError(f"{what}_block_scales have shape {tuple(scales.shape)}, need "
                         f"{(*shape[:3], shape[3] // 16)}")
    ps, ss = pages.stride(), scales.stride()
    if ss[3] != 1 or any(n > 1 and p != 16 * b for n, p, b in zip(shape[:3], ps, ss)):
        raise ValueError(f"{what}_block_scales must be laid out as the pages: strides of a 16th of theirs "
                         f"({ps[:3]}), not {ss[:3]}, and contiguous rows")
    return scales.data_ptr()


def _kv_cache(k_pages, v_pages, k_scale, v_scale, k_block_scales=None, v_block_scales=None):
    """bitdelta_kv_cache of two [pages, page_size, kv_heads, head_dim] tensors (bf16 or
    float8_e4m3fn; uint8, two 4-bit codes each, [.., head_dim / 2]), any strides but contiguous rows."""
    import torch
    if not _KV_DTYPES:
        _KV_DTYPES.update({torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.uint8: 2})
    for t, what in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what} must be a CUDA/HIP torch tensor")
    shape, dtype = k_pages.shape, k_pages.dtype
    code = _KV_DTYPES.get(dtype)
    if code is None or v_pages.dtype is not dtype:
        raise TypeError("k_pages and v_pages must both be torch.bfloat16, torch.float8_e4m3fn or (4 bits) "
                        f"torch.uint8, got {dtype} and {v_pages.dtype}")
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [pages, page_size, kv_heads, head_dim], "
                         "of one shape")
    ks, vs = k_pages.stride(), v_pages.stride()
    if shape[3] > 1 and (ks[3] != 1 or vs[3] != 1):
        raise ValueError("k_pages and v_pages must have contiguous rows")
    device = k_pages.device
    if v_pages.device != device:
        raise ValueError(f"v_pages are on {v_pages.device}, k_pages on {device}")
    if code != 2:
        if k_block_scales is not None or v_block_scales is not None:
            raise ValueError(f"pages of {dtype} have no block scales")
        return _KvCache(k_pages.data_ptr(), v_pages.data_ptr(), code, shape[0], shape[1], shape[2],
                        shape[3], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], k_scale, v_scale)
    # the usual case in one test each (0.4 instead of 1.3 us of a call of some 10)
    want, u8, blocks = (shape[0], shape[1], shape[2], shape[3] >> 4), torch.uint8, []
    for pages, strides, scales, what in ((k_pages, ks, k_block_scales, "k"),
                                         (v_pages, vs, v_block_scales, "v")):
        if not (isinstance(scales, torch.Tensor) and scales.dtype is u8 and scales.device == device
                and scales.shape == want
                and scales.stride() == (strides[0] / 16, strides[1] / 16, strides[2] / 16, 1)):
            blocks.append(_block_scales(pages, scales, what))
        else:
            blocks.append(scales.data_ptr())
    return _KvCache(k_pages.data_ptr(), v_pages.data_ptr(), 2, shape[0], shape[1], shape[2],
                    2 * shape[3], 2 * ks[0], 2 * ks[1], 2 * ks[2], 2 * vs[0], 2 * vs[1], 2 * vs[2],
                    k_scale, v_scale, blocks[0], blocks[1])


def _cache_sizes(k_pages):
    """The same for a query of workspace sizes: no scales are looked at."""
    import torch
    if not isinstance(k_pages, torch.Tensor) or not k_pages.is_cuda or k_pages.dtype is not torch.uint8:
        return _kv_cache(k_pages, k_pages, 1.0, 1.0)
    shape, ks = k_pages.shape, k_pages.stride()
    if len(shape) != 4:
        raise ValueError("k_pages must be [pages, page_size, kv_heads, head_dim / 2]")
    p = k_pages.data_ptr()
    return _KvCache(p, p, 2, shape[0], shape[1], shape[2], 2 * shape[3], *[2 * x for x in ks[:3]],
                    *[2 * x for x in ks[:3]], 1.0, 1.0, p, p)


def _attend_rows(q, cache, out, lse, return_lse, scale, stream):
    """(bitdelta_attend_rows, out, lse) for q [tokens, heads, head_dim]; out and lse are made here
    when missing."""
    import torch
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA/HIP torch tensor")
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"q must be torch.bfloat16, got {q.dtype}")
    shape, dim = q.shape, cache.head_dim
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"q must be [tokens, heads, {dim}], not {tuple(shape)}")
    qs = q.stride()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None else \
            _empty(shape, q.dtype, q.device, stream)
    elif not out.is_cuda or out.dtype is not torch.bfloat16:
        raise TypeError("out must be a torch.bfloat16 CUDA/HIP tensor")
    elif out.shape != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, needs {tuple(shape)}")
    os_ = out.stride()
    if qs[2] != 1 or os_[2] != 1:
        raise ValueError("q and out must have contiguous rows")
    lptr = None
    if lse is not None:
        _check_shape(lse, shape[:2], "lse")
        lptr = _dev(lse, "torch.float32", "lse")
    elif return_lse:
        lse = torch.empty(shape[0], shape[1], dtype=torch.float32, device=q.device) if stream is None else \
            _empty(shape[:2], torch.float32, q.device, stream)
        lptr = lse.data_ptr()
    return _AttendRows(q.data_ptr(), out.data_ptr(), lptr, shape[0], shape[1], qs[0], qs[1], os_[0],
                       os_[1], dim ** -0.5 if scale is None else scale), out, lse


def _table(t, lens, n, what):
    """(pointer, width, lens pointer) of an int32 page table [n, width] and its lengths [n]."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError(f"{what} must be [{n}, pages], not {tuple(shape)}")
    if lens.dim() != 1 or lens.shape[0] != n:
        raise ValueError(f"{what}'s lengths must be [{n}], not {tuple(lens.shape)}")
    return _dev(t, "torch.int32", what), shape[1], _dev(lens, "torch.int32", what + "'s lengths")


def _host_i32(a):
    """(array, its address) of a host int32 array."""
    arr = np.ascontiguousarray(a, dtype=np.int32)
    return arr, arr.__array_interface__["data"][0]


def attend_shared_workspace_bytes(k_pages, heads, table, prefix_table, seg_offsets) -> int:
    """Device workspace an attend_shared call with these tables needs (bytes, 0 if none)."""
    offs, offs_p = _host_i32(seg_offsets)
    c = _cache_sizes(k_pages)
    pwidth = 0 if prefix_table is None else int(prefix_table.shape[1])
    return int(_lib().bitdelta_attend_shared_workspace_bytes(
        int(table.shape[0]), heads, ctypes.byref(c), int(table.shape[1]), pwidth, offs_p,
        offs.size - 1))


def attend_shared(q, k_pages, v_pages, table, lens, prefix_table, prefix_lens, seg_offsets,
                  scale=None, k_scale=1.0, v_scale=1.0, out=None, lse=None, return_lse=False,
                  workspace=None, stream=None, k_block_scales=None, v_block_scales=None):
    """Decode attention, one new token per sequence, over a paged cache whose prefixes are shared
    by segment: sequence b of segment g (``seg_offsets`` as plan_segments returns them) sees the
    first ``prefix_lens[g]`` tokens of ``prefix_table[g]``, then the first ``lens[b]`` of
    ``table[b]``.

    ``q``: bf16 [batch, heads, head_dim]; ``k_pages`` / ``v_pages``: [pages, page_size, kv_heads,
    head_dim] bf16 or float8_e4m3fn (each stored value times ``k_scale`` / ``v_scale``), any
    strides but contiguous rows, or 4-bit pages with their block scales (see cache_write); ``table``
    int32 [batch, n], ``lens`` int32 [batch], ``prefix_table`` int32 [segments, m] and
    ``prefix_lens`` int32 [segments] (both None: no prefixes), on the device.  Returns bf16 ``out``
    like q, and with ``return_lse`` (or ``lse`` given) also the natural log of each row's softmax
    sum, float32 [batch, heads].  A sequence with no keys gives zeros and -inf."""
    offs, offs_p = _host_i32(seg_offsets)
    cache = _kv_cache(k_pages, v_pages, k_scale, v_scale, k_block_scales, v_block_scales)
    rows, out, lse = _attend_rows(q, cache, out, lse, return_lse, scale, stream)
    tptr, width, lptr = _table(table, lens, rows.tokens, "table")
    if offs.size < 1:
        raise ValueError("seg_offsets must hold at least one offset")
    nseg = offs.size - 1
    if (prefix_table is None) != (prefix_lens is None):
        raise ValueError("give prefix_table and prefix_lens, or neither")
    pptr, pwidth, plptr = None, 0, None
    if prefix_table is not None:
        pptr, pwidth, plptr = _table(prefix_table, prefix_lens, nseg, "prefix_table")
    need = 0 if workspace is not None else int(_lib().bitdelta_attend_shared_workspace_bytes(
        rows.tokens, rows.heads, ctypes.byref(cache), width, pwidth, offs_p, nseg))
    ws_ptr, ws_bytes, ws = _workspace(workspace, need, q.device, stream)
    _check(_lib().bitdelta_attend_shared(
        ctypes.byref(rows), ctypes.byref(cache), tptr, width, lptr, pptr, pwidth, plptr, offs_p,
        nseg, ws_ptr, ws_bytes, _raw_stream(stream, q)), "bitdelta_attend_shared")
    return out if lse is None else (out, lse)


def attend_window_workspace_bytes(k_pages, heads, table, tokens, max_q_len, window, sinks) -> int:
    """Device workspace an attend_window call of these sizes needs (bytes, 0 if none)."""
    c = _cache_sizes(k_pages)
    return int(_lib().bitdelta_attend_window_workspace_bytes(
        tokens, heads, ctypes.byref(c), int(table.shape[0]), int(table.shape[1]), max_q_len,
        window, sinks))


def attend_window(q, k_pages, v_pages, table, lens, window, sinks=0, q_offsets=None, max_q_len=None,
                  scale=None, k_scale=1.0, v_scale=1.0, out=None, lse=None, return_lse=False,
                  workspace=None, stream=None, k_block_scales=None, v_block_scales=None):
    """Causal attention of each sequence's last tokens over a paged cache, with a sliding window
    and first tokens that stay visible: the token at position p sees key j iff j <= p and
    (p - j < ``window`` or j < ``sinks``).  Sequence b holds ``lens[b]`` keys, its new tokens
    among them as the last ones.

    ``q``: bf16 [tokens, heads, head_dim]; sequence b's rows are q_offsets[b] .. q_offsets[b + 1]
    (int32 [batch + 1] on the device; None: one token per sequence).  ``max_q_len`` is at least the
    longest chunk (None: 1 without q_offsets, else the number of tokens; the real length picks better
    kernels); a chunk's rows beyond its first ``max_q_len`` are not computed.  Cache, tables, scales
    and results as for attend_shared."""
    cache = _kv_cache(k_pages, v_pages, k_scale, v_scale, k_block_scales, v_block_scales)
    rows, out, lse = _attend_rows(q, cache, out, lse, return_lse, scale, stream)
    batch = lens.shape[0] if lens.dim() == 1 else -1
    tptr, width, lptr = _table(table, lens, batch, "table")
    optr = None
    if max_q_len is None:
        max_q_len = 1 if q_offsets is None else max(rows.tokens, 1)
    if q_offsets is not None:
        _check_shape(q_offsets, (batch + 1,), "q_offsets")
        optr = _dev(q_offsets, "torch.int32", "q_offsets")
    need = 0 if workspace is not None else int(_lib().bitdelta_attend_window_workspace_bytes(
        rows.tokens, rows.heads, ctypes.byref(cache), batch, width, max_q_len, window, sinks))
    ws_ptr, ws_bytes, ws = _workspace(workspace, need, q.device, stream)
    _check(_lib().bitdelta_attend_window(
        ctypes.byref(rows), ctypes.byref(cache), batch, tptr, width, lptr, optr, max_q_len, window,
        sinks, ws_ptr, ws_bytes, _raw_stream(stream, q)), "bitdelta_attend_window")
    return out if lse is None else (out, lse)


# ---------------------------------------------------------------------------------------------
# Writing and reading the paged cache
# ---------------------------------------------------------------------------------------------

def _kv_rows(k, v, cache, device):
    """bitdelta_kv_rows of two bf16 [tokens, kv_heads, head_dim] tensors."""
    import torch
    bf16 = torch.bfloat16
    for t, what in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what} must be a CUDA/HIP torch tensor")
        if t.dtype is not bf16:
            raise TypeError(f"{what} must be torch.bfloat16, got {t.dtype}")
        if t.device != device:
            raise ValueError(f"{what} is on {t.device}, the pages on {device}")
    shape = k.shape
    if len(shape) != 3 or shape[1] != cache.kv_heads or shape[2] != cache.head_dim or v.shape != shape:
        raise ValueError(f"k and v must be [tokens, {cache.kv_heads}, {cache.head_dim}], not "
                         f"{tuple(shape)} and {tuple(v.shape)}")
    ks, vs = k.stride(), v.stride()
    if shape[0] and (ks[2] != 1 or vs[2] != 1):
        raise ValueError("k and v must have contiguous rows")
    return _KvRows(k.data_ptr(), v.data_ptr(), shape[0], ks[0], ks[1], vs[0], vs[1])


def _cache_places(table, lens, q_offsets, device):
    """(batch, table pointer, width, lens pointer, q_offsets pointer)."""
    import torch
    i32 = torch.int32
    # the usual case in one test, as above
    if isinstance(table, torch.Tensor) and isinstance(lens, torch.Tensor) and table.dtype is i32 \
            and lens.dtype is i32 and table.device == device and lens.device == device \
            and table.dim() == 2 and lens.dim() == 1 and table.is_contiguous() and lens.is_contiguous() \
            and table.shape[0] == lens.shape[0]:
        batch, width = table.shape
        tptr, lptr = table.data_ptr(), lens.data_ptr()
    else:
        batch = lens.shape[0] if lens.dim() == 1 else -1
        tptr, width, lptr = _table(table, lens, batch, "table")
    optr = None
    if q_offsets is not None:
        _check_shape(q_offsets, (batch + 1,), "q_offsets")
        optr = _dev(q_offsets, "torch.int32", "q_offsets")
    if table.device != device or lens.device != device or (optr and q_offsets.device != device):
        raise ValueError(f"table, lens and q_offsets must be on {device}, as the pages")
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"the pages are on {device}, which is not the current device")
    return batch, tptr, width, lptr, optr


def cache_write(k, v, k_pages, v_pages, table, lens, q_offsets=None, k_scale=1.0, v_scale=1.0,
                k_block_scales=None, v_block_scales=None, stream=None):
    """New keys and values into their pages, quantised on the way.  Which token a row is goes by the
    tables as attend_window has them: sequence b holds ``lens[b]`` tokens, its new ones among them as the
    last ones, which are rows q_offsets[b] .. q_offsets[b + 1] (int32 [batch + 1] on the device; None: one
    token per sequence).  Rows whose token has no page in the table are not written (a length beyond the
    table is not cut to what it holds, as the attentions cut it).

    ``k`` / ``v``: bf16 [tokens, kv_heads, head_dim], contiguous rows.  ``k_pages`` / ``v_pages``:
    [pages, page_size, kv_heads, head_dim] bf16 or float8_e4m3fn, which get each value divided by
    ``k_scale`` / ``v_scale`` and rounded (float8: at most +-448), or, in 4 bits, uint8 [..., head_dim /
    2] with ``k_block_scales`` / ``v_block_scales``, uint8 [..., head_dim / 32] of a 16th of the pages'
    strides: each 32 values of a row share a power of two, byte - 127, such that the largest is at most 7
    of them, and are rounded to 0, 0.5, 1, 1.5, 2, 3, 4 or 6 of them (lower four bits first).  Infinities
    and NaN stay what they are in bf16; in float8 they become NaN, in 4 bits their whole block.  Returns
    (k_pages, v_pages)."""
    cache = _kv_cache(k_pages, v_pages, k_scale, v_scale, k_block_scales, v_block_scales)
    device = k_pages.device
    rows = _kv_rows(k, v, cache, device)
    batch, tptr, width, lptr, optr = _cache_places(table, lens, q_offsets, device)
    _check(_lib().bitdelta_cache_write(ctypes.byref(rows), ctypes.byref(cache), batch, tptr, width, lptr,
                                       optr, _raw_stream(stream, k_pages)), "bitdelta_cache_write")
    return k_pages, v_pages


def cache_read(k_pages, v_pages, table, lens, q_offsets=None, tokens=None, k_scale=1.0, v_scale=1.0,
               k_block_scales=None, v_block_scales=None, k_out=None, v_out=None, stream=None):
    """The rows cache_write wrote by these tables, read back: bf16 (k, v) [tokens, kv_heads, head_dim],
    each stored value times ``k_scale`` / ``v_scale``.  With q_offsets, ``tokens`` (or ``k_out`` and
    ``v_out``) says how many rows there are; q_offsets that begin at 0 and rise by ``lens`` read whole
    sequences.  Tokens without a page are zeros; rows of no sequence stay as they are in k_out and v_out
    (in results made here: anything)."""
    import torch
    cache = _kv_cache(k_pages, v_pages, k_scale, v_scale, k_block_scales, v_block_scales)
    device = k_pages.device
    batch, tptr, width, lptr, optr = _cache_places(table, lens, q_offsets, device)
    if (k_out is None) != (v_out is None):
        raise ValueError("give k_out and v_out, or neither")
    if k_out is None:
        if tokens is None:
            if q_offsets is not None:
                raise ValueError("with q_offsets, give tokens or k_out and v_out")
            tokens = batch
        shape = (2, tokens, cache.kv_heads, cache.head_dim)
        both = torch.empty(shape, dtype=torch.bfloat16, device=device) if stream is None else \
            _empty(shape, torch.bfloat16, device, stream)
        k_out, v_out = both.unbind(0)
    elif tokens is not None and k_out.shape[:1] != (tokens,):
        raise ValueError(f"k_out has shape {tuple(k_out.shape)}, needs {tokens} tokens")
    rows = _kv_rows(k_out, v_out, cache, device)
    _check(_lib().bitdelta_cache_read(ctypes.byref(rows), ctypes.byref(cache), batch, tptr, width, lptr,
                                      optr, _raw_stream(stream, k_pages)), "bitdelta_cache_read")
    return k_out, v_out


# ---------------------------------------------------------------------------------------------
# Sampling
# ---------------------------------------------------------------------------------------------

def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, logprob=None,
           return_logprob=False, stream=None):
    """The next token of each row of ``logits`` ([rows, vocab], bf16 or float32, contiguous rows)
    from the uniform numbers ``u`` (float32 [rows] in [0, 1)).  Tokens are ordered by descending
    logit, ties by index; ``top_k`` (int32 [rows], <= 0: off), ``top_p`` and ``min_p`` (float32
    [rows], >= 1 and <= 0: off) each keep a prefix of that order, weighed by
    exp((logit - largest) / ``temperature``) (float32 [rows]; 0: the first token); the token drawn
    is the first whose running weight exceeds u times the kept weight.  Returns int32 [rows] (-1:
    every logit is -inf), and with ``return_logprob`` (or ``logprob`` given) also the natural log
    of the token's share of the kept weight, float32 [rows]."""
    import torch
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA/HIP torch tensor")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = (int(n) for n in logits.shape)
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits must have contiguous rows")
    stride = int(logits.stride(0)) if rows > 1 else max(int(logits.stride(0)), vocab)

    want = logits.shape[:1]

    def arg(t, dtype, what):
        if t is None:
            return None
        if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == want \
                and t.is_contiguous():
            return t.data_ptr()
        _check_shape(t, want, what)
        return _dev(t, str(dtype), what)

    f32, i32 = torch.float32, torch.int32
    if out is None:
        out = torch.empty(rows, dtype=i32, device=logits.device) if stream is None else \
            _empty(rows, i32, logits.device, stream)
    if logprob is None and return_logprob:
        logprob = torch.empty(rows, dtype=f32, device=logits.device) if stream is None else \
            _empty(rows, f32, logits.device, stream)
    _check(_lib().bitdelta_sample(
        logits.data_ptr(), 0 if logits.dtype == torch.bfloat16 else 1, rows, vocab, stride,
        arg(u, f32, "u"), arg(temperature, f32, "temperature"), arg(top_k, i32, "top_k"),
        arg(top_p, f32, "top_p"), arg(min_p, f32, "min_p"), arg(out, i32, "out"),
        arg(logprob, f32, "logprob"), _raw_stream(stream, logits)), "bitdelta_sample")
    return out if logprob is None else (out, logprob)
