"""ctypes binding over libpagedkv.so (see include/pagedkv.h for the C ABI).

Argument marshalling only: every step of append and decode runs in the library's CUDA
kernels. PyTorch supplies device memory (outputs and the workspace come from its
caching allocator) and the current CUDA stream. There is no fallback: if the library
is missing or a tensor is not on a CUDA device, the call raises.
"""

from __future__ import annotations

import ctypes
import enum
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.environ.get("PAGEDKV_LIB", os.path.join(_HERE, "libpagedkv.so"))


class Status(enum.IntEnum):
    OK = 0
    ERR_NULL = -1
    ERR_DTYPE = -2
    ERR_SHAPE = -3
    ERR_UNSUPPORTED = -4
    ERR_WORKSPACE = -5
    ERR_CUDA = -6
    ERR_ALIGNMENT = -7
    ERR_HOST_MEMORY = -8


DEV_BAD_CONTEXT_LEN = 0x1
DEV_BAD_BLOCK_ID = 0x2
DEV_TIMEOUT = 0x4
DEV_BAD_PREFIX = 0x8
DEV_BAD_POSITION = 0x10
DEV_NO_BLOCKS = 0x20

KV_BF16 = 0
KV_INT8 = 1
KV_FP8_E4M3 = 2
KV_FP8_E5M2 = 3
FP8_FORMATS = {"e4m3": KV_FP8_E4M3, "e5m2": KV_FP8_E5M2}


_KV_OF_DTYPE = {torch.bfloat16: KV_BF16, torch.int8: KV_INT8, torch.uint8: None,
                torch.float8_e4m3fn: KV_FP8_E4M3, torch.float8_e5m2: KV_FP8_E5M2}


class PagedKVError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib().pkv_status_string(status).decode()}")


class Dims(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32)]


class Rotary(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("num_positions", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float)]


EXPORTS = {
    "pkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pkv_version": (ctypes.c_int, []),
    "pkv_kernel_launch_count": (ctypes.c_uint64, []),
    "pkv_append_bf16": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int32, ctypes.c_void_p,
                                                                ctypes.c_void_p]),
    "pkv_append_int8": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_int32, ctypes.c_void_p,
                                                                ctypes.c_void_p]),
    "pkv_decode_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int,
                                                  ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_bf16": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_float, ctypes.c_void_p,
                                                                ctypes.c_void_p, ctypes.c_size_t,
                                                                ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_decode_int8": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_float, ctypes.c_void_p,
                                                                ctypes.c_void_p, ctypes.c_size_t,
                                                                ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_append_fp8": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_int32, ctypes.c_int,
                                                               ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_decode_fp8": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_float, ctypes.c_int,
                                                               ctypes.c_void_p, ctypes.c_void_p,
                                                               ctypes.c_size_t, ctypes.c_void_p,
                                                               ctypes.c_void_p]),
    "pkv_rotate_append_bf16": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int32] +
                               [ctypes.c_void_p] * 3),
    "pkv_rotate_append_q8": (ctypes.c_int, [ctypes.c_void_p] * 11 + [ctypes.c_int32,
                                                                     ctypes.c_int] +
                             [ctypes.c_void_p] * 3),
    "pkv_gather_tokens": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int32, ctypes.c_int] +
                          [ctypes.c_void_p] * 3),
    "pkv_decode_diff_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int,
                                                       ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_diff_bf16": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_float] * 3 +
                             [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                              ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_decode_diff_q8": (ctypes.c_int, [ctypes.c_void_p] * 10 + [ctypes.c_float] * 3 +
                           [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                            ctypes.c_void_p, ctypes.c_void_p]),
    "pkv_resize_sequences": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int32] +
                             [ctypes.c_void_p] * 3 + [ctypes.c_int32] + [ctypes.c_void_p] * 3),
    "pkv_keep_tokens": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_int32, ctypes.c_int] +
                        [ctypes.c_void_p] * 3),
    "pkv_decode_tree_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32,
                                                       ctypes.c_int,
                                                       ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_tree_bf16": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_int32,
                                                                    ctypes.c_float,
                                                                    ctypes.c_void_p,
                                                                    ctypes.c_void_p,
                                                                    ctypes.c_size_t,
                                                                    ctypes.c_void_p,
                                                                    ctypes.c_void_p]),
    "pkv_decode_tree_q8": (ctypes.c_int, [ctypes.c_void_p] * 10 + [ctypes.c_int32,
                                                                   ctypes.c_float, ctypes.c_int,
                                                                   ctypes.c_void_p,
                                                                   ctypes.c_void_p,
                                                                   ctypes.c_size_t,
                                                                   ctypes.c_void_p,
                                                                   ctypes.c_void_p]),
    "pkv_prompt_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p,
                                                  ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_prompt_attention_bf16": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_float,
                                                                         ctypes.c_void_p,
                                                                         ctypes.c_void_p,
                                                                         ctypes.c_size_t,
                                                                         ctypes.c_void_p,
                                                                         ctypes.c_void_p]),
    "pkv_copy_blocks": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_int32, ctypes.c_int,
                                                                ctypes.c_void_p, ctypes.c_void_p,
                                                                ctypes.c_void_p]),
    "pkv_swap_out": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int32, ctypes.c_int,
                                                             ctypes.c_void_p, ctypes.c_void_p,
                                                             ctypes.c_void_p]),
    "pkv_swap_in": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int32, ctypes.c_int,
                                                            ctypes.c_void_p, ctypes.c_void_p,
                                                            ctypes.c_void_p]),
    "pkv_decode_multi_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32,
                                                        ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_multi_bf16": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_int32,
                                                                      ctypes.c_float,
                                                                      ctypes.c_void_p,
                                                                      ctypes.c_void_p,
                                                                      ctypes.c_size_t,
                                                                      ctypes.c_void_p,
                                                                      ctypes.c_void_p]),
    "pkv_decode_multi_q8_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32,
                                                           ctypes.c_int,
                                                           ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_multi_q8": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_int32,
                                                                   ctypes.c_float, ctypes.c_int,
                                                                   ctypes.c_void_p,
                                                                   ctypes.c_void_p,
                                                                   ctypes.c_size_t,
                                                                   ctypes.c_void_p,
                                                                   ctypes.c_void_p]),
    "pkv_decode_cascade_q8_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32,
                                                             ctypes.c_int,
                                                             ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_cascade_q8": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_int32,
                                                                     ctypes.c_float, ctypes.c_int,
                                                                     ctypes.c_void_p,
                                                                     ctypes.c_void_p,
                                                                     ctypes.c_size_t,
                                                                     ctypes.c_void_p,
                                                                     ctypes.c_void_p]),
    "pkv_decode_cascade_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32,
                                                          ctypes.POINTER(ctypes.c_size_t)]),
    "pkv_decode_cascade_bf16": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_int32,
                                                                        ctypes.c_float,
                                                                        ctypes.c_void_p,
                                                                        ctypes.c_void_p,
                                                                        ctypes.c_size_t,
                                                                        ctypes.c_void_p,
                                                                        ctypes.c_void_p]),
    "pkv_decode_bf16_noalloc": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_float,
                                                                        ctypes.c_void_p,
                                                                        ctypes.c_void_p,
                                                                        ctypes.c_void_p]),
}

_LIB = None
_LOCK = threading.Lock()


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libpagedkv.so (raises if it has not been built)."""
    global _LIB
    with _LOCK:
        if _LIB is not None and path is None:
            return _LIB
        p = path or library_path()
        if not os.path.exists(p):
            raise ImportError(f"{p} not found: build it with `python -m "
                              f"paged_kv_decode_02_gb300.build_lib` (there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _LIB = lib
        return lib


def _lib():
    return _LIB if _LIB is not None else load_library()


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


class _OnDevice:
    """Make `device` current for the library call (a no-op when it already is)."""

    __slots__ = ("dev", "prev")

    def __init__(self, device):
        self.dev = device.index if device.index is not None else torch.cuda.current_device()
        self.prev = None

    def __enter__(self):
        cur = torch.cuda.current_device()
        if cur != self.dev:
            self.prev = cur
            torch.cuda.set_device(self.dev)

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _check(status, what):
    if status != 0:
        raise PagedKVError(status, what)


def _require(t, name, dtype, ndim, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


# ---------------------------------------------------------------------------
# Lean marshalling: a small decode step is a few microseconds on the GPU, so the calls
# below check and pass their arguments with as little Python as that takes. Pointers go as
# integers, the C structs as packed bytes; _need() looks at a tensor through four cheap
# accessors and leaves the wording of a refusal to _require().
# ---------------------------------------------------------------------------
_pack_dims = struct.Struct("7i").pack                  # pkv_dims
_pack_rotary = struct.Struct("3P4q3if").pack           # pkv_rotary
_pack_prompt = struct.Struct("6i4q").pack              # pkv_prompt_dims
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_Tensor = torch.Tensor
_current_device = getattr(torch._C, "_cuda_getDevice", None)      # (None: torch without CUDA)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_CACHE_DTYPES = {KV_BF16: (torch.bfloat16,), KV_INT8: (torch.int8,),
                 KV_FP8_E4M3: (torch.uint8, torch.float8_e4m3fn),
                 KV_FP8_E5M2: (torch.uint8, torch.float8_e5m2)}


def _need(t, name, dtype, ndim, index):
    """:func:`_require` of a tensor on CUDA device ``index``."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index
            and t.dim() == ndim and t.is_contiguous()):
        _require(t, name, dtype, ndim, torch.device("cuda", max(index, 0)))


def _need_caches(kv, k_cache, v_cache, k_scale, v_scale):
    """Checks the caches of a KV dtype; returns (device index, K cache's shape)."""
    if not isinstance(k_cache, _Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    index = k_cache.get_device()
    if index < 0:
        _require(k_cache, "k_cache", k_cache.dtype, 4)
    dt = k_cache.dtype
    if dt not in _CACHE_DTYPES[kv]:
        dt = _CACHE_DTYPES[kv][0]
    _need(k_cache, "k_cache", dt, 4, index)
    shape = k_cache.shape
    if not (isinstance(v_cache, _Tensor) and v_cache.dtype is dt
            and v_cache.get_device() == index and v_cache.shape == shape
            and v_cache.is_contiguous()):
        _require_any(v_cache, "v_cache", _code_dtypes(kv), 4, k_cache.device)
        _same_shape(v_cache, "v_cache", shape)
    if kv != KV_BF16:
        _need(k_scale, "k_scale", _F32, 3, index)
        _need(v_scale, "v_scale", _F32, 3, index)
        if k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
            _cache_shapes(k_cache, v_cache, k_scale, v_scale)
    return index, shape


def _run(name, index, *args):
    """Calls the library on CUDA device ``index``, on its current stream; returns the
    status."""
    fn = getattr(_LIB if _LIB is not None else load_library(), name)
    if _current_device() == index:
        return fn(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return fn(*args, _raw_stream(index))


def _status_ptr(status, index):
    if status is None:
        return None
    return _status_word(status, torch.device("cuda", index)).data_ptr()


def _dims(num_seqs, num_q_heads, k_cache, max_blocks_per_seq):
    nb, hkv, bs, d = k_cache.shape
    return Dims(num_seqs, num_q_heads, hkv, d, bs, nb, max_blocks_per_seq)


def _same_shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _cache_shapes(k_cache, v_cache, k_scale=None, v_scale=None):
    """V cache and scales against the K cache [NB, Hkv, bs, D]: the kernels address all
    of them through the K cache's sizes."""
    _same_shape(v_cache, "v_cache", k_cache.shape)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is not None:
            _same_shape(t, n, k_cache.shape[:3])


def _append_shapes(k, v, k_cache, v_cache, slot_mapping, k_scale=None, v_scale=None):
    """New rows [T, Hkv, D] and T slots, against the caches."""
    _cache_shapes(k_cache, v_cache, k_scale, v_scale)
    row = (k.shape[0], k_cache.shape[1], k_cache.shape[3])
    _same_shape(k, "k", row)
    _same_shape(v, "v", row)
    _same_shape(slot_mapping, "slot_mapping", (k.shape[0],))


def paged_kv_append(k, v, k_cache, v_cache, slot_mapping):
    """Write new tokens' K/V rows ([T, Hkv, D] bf16) into the bf16 paged caches
    ([NB, Hkv, bs, D]) at ``slot_mapping`` ([T] int64, -1 = skip). In place."""
    dev = k_cache.device
    for t, n, dt, nd in ((k, "k", torch.bfloat16, 3), (v, "v", torch.bfloat16, 3),
                         (k_cache, "k_cache", torch.bfloat16, 4),
                         (v_cache, "v_cache", torch.bfloat16, 4),
                         (slot_mapping, "slot_mapping", torch.int64, 1)):
        _require(t, n, dt, nd, dev)
    _append_shapes(k, v, k_cache, v_cache, slot_mapping)
    dims = _dims(0, k_cache.shape[1], k_cache, 1)
    with _OnDevice(dev):
        st = _lib().pkv_append_bf16(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(slot_mapping), k.shape[0], ctypes.byref(dims),
                                    _stream(dev))
    _check(st, "pkv_append_bf16")


def paged_kv_append_int8(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping):
    """Quantise new tokens' K/V rows per (token, KV head) and write INT8 codes into
    ``k_cache``/``v_cache`` ([NB, Hkv, bs, D] int8) and fp32 scales into
    ``k_scale``/``v_scale`` ([NB, Hkv, bs]). In place."""
    dev = k_cache.device
    for t, n, dt, nd in ((k, "k", torch.bfloat16, 3), (v, "v", torch.bfloat16, 3),
                         (k_cache, "k_cache", torch.int8, 4), (v_cache, "v_cache", torch.int8, 4),
                         (k_scale, "k_scale", torch.float32, 3),
                         (v_scale, "v_scale", torch.float32, 3),
                         (slot_mapping, "slot_mapping", torch.int64, 1)):
        _require(t, n, dt, nd, dev)
    _append_shapes(k, v, k_cache, v_cache, slot_mapping, k_scale, v_scale)
    dims = _dims(0, k_cache.shape[1], k_cache, 1)
    with _OnDevice(dev):
        st = _lib().pkv_append_int8(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping), k.shape[0],
                                    ctypes.byref(dims), _stream(dev))
    _check(st, "pkv_append_int8")


def paged_kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, fmt="e5m2"):
    """Quantise new tokens' K/V rows per (token, KV head) to FP8 (``fmt`` "e4m3" or
    "e5m2") and write the codes into ``k_cache``/``v_cache`` ([NB, Hkv, bs, D] uint8 or
    the matching torch float8 dtype) and fp32 scales into ``k_scale``/``v_scale``
    ([NB, Hkv, bs]). In place."""
    kv = _fp8_format(fmt)
    dev = k_cache.device
    for t, n, dt, nd in ((k, "k", torch.bfloat16, 3), (v, "v", torch.bfloat16, 3),
                         (k_scale, "k_scale", torch.float32, 3),
                         (v_scale, "v_scale", torch.float32, 3),
                         (slot_mapping, "slot_mapping", torch.int64, 1)):
        _require(t, n, dt, nd, dev)
    _require_any(k_cache, "k_cache", _code_dtypes(kv), 4, dev)
    _require_any(v_cache, "v_cache", _code_dtypes(kv), 4, dev)
    _append_shapes(k, v, k_cache, v_cache, slot_mapping, k_scale, v_scale)
    dims = _dims(0, k_cache.shape[1], k_cache, 1)
    with _OnDevice(dev):
        st = _lib().pkv_append_fp8(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping), k.shape[0],
                                   kv, ctypes.byref(dims), _stream(dev))
    _check(st, "pkv_append_fp8")


def _token_rows(t, name, index):
    """Checks a [T, H, D] bf16 tensor of contiguous rows of heads; returns its shape and its
    token stride (any, as of a slice of a fused projection's output)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == index
            and t.dim() == 3):
        _require(t, name, _BF16, 3, torch.device("cuda", max(index, 0)))
    shape = t.shape
    tokens, heads, d = shape
    st0, st1, st2 = t.stride()
    if (d > 1 and st2 != 1) or (heads > 1 and st1 != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous rows")
    return shape, st0 if tokens > 1 else heads * d


def _rotate_append(kv, q, k, v, positions, cos_sin, k_cache, v_cache, k_scale, v_scale,
                   slot_mapping, q_norm, k_norm, eps, interleaved, out, status):
    index, (nb, hkv, bs, d) = _need_caches(kv, k_cache, v_cache, k_scale, v_scale)
    q_shape, q_stride = _token_rows(q, "q", index)
    k_shape, k_stride = _token_rows(k, "k", index)
    v_shape, v_stride = _token_rows(v, "v", index)
    tokens, hq, dq = q_shape
    if dq != d:
        raise ValueError("cache shapes disagree with q")
    if k_shape != (tokens, hkv, d) or v_shape != k_shape:
        _same_shape(k, "k", (tokens, hkv, d))
        _same_shape(v, "v", (tokens, hkv, d))
    _need(positions, "positions", _I64, 1, index)
    _need(slot_mapping, "slot_mapping", _I64, 1, index)
    _need(cos_sin, "cos_sin", _F32, 2, index)
    if positions.shape[0] != tokens or slot_mapping.shape[0] != tokens:
        _same_shape(positions, "positions", (tokens,))
        _same_shape(slot_mapping, "slot_mapping", (tokens,))
    qw = kw = 0
    if q_norm is not None:
        _need(q_norm, "q_norm", _BF16, 1, index)
        qw = q_norm.data_ptr()
    if k_norm is not None:
        _need(k_norm, "k_norm", _BF16, 1, index)
        kw = k_norm.data_ptr()
    if (qw and q_norm.shape[0] != d) or (kw and k_norm.shape[0] != d):
        raise ValueError(f"q_norm and k_norm must have {d} elements")
    if out is None:
        out, out_stride = torch.empty((tokens, hq, d), dtype=_BF16, device=q.device), hq * d
    else:
        out_shape, out_stride = _token_rows(out, "out", index)
        if out_shape != q_shape:
            _same_shape(out, "out", q_shape)
    rotary = _pack_rotary(cos_sin.data_ptr(), qw, kw, out_stride, q_stride, k_stride, v_stride,
                          *cos_sin.shape, 1 if interleaved else 0, float(eps))
    dims = _pack_dims(0, hq, hkv, d, bs, nb, 1)
    rows = (out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(),
            rotary, k_cache.data_ptr(), v_cache.data_ptr())
    status = _status_ptr(status, index)
    if kv == KV_BF16:
        name = "pkv_rotate_append_bf16"
        st = _run(name, index, *rows, slot_mapping.data_ptr(), tokens, dims, status)
    else:
        name = "pkv_rotate_append_q8"
        st = _run(name, index, *rows, k_scale.data_ptr(), v_scale.data_ptr(),
                  slot_mapping.data_ptr(), tokens, kv, dims, status)
    if st:
        _check(st, name)
    return out


def paged_kv_rotate_append(q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping,
                           q_norm=None, k_norm=None, eps=1e-6, interleaved=False, out=None,
                           status=None):
    """Norm and rotate new tokens' queries and keys and write K and V into the bf16 paged
    caches, in one pass.

    q [T, Hq, D], k and v [T, Hkv, D] bf16 (any token stride that is a multiple of 8, as
    slices of a fused projection have); positions [T] int64; cos_sin [positions, R] fp32,
    R / 2 cosines then R / 2 sines per position, R the rotated part of a row (a multiple of
    16, at most D): element i turns with i + R / 2, or 2i with 2i + 1 (``interleaved``).
    ``q_norm`` / ``k_norm`` ([D] bf16): root-mean-square norm weights of each head's row
    (None: no norm). ``slot_mapping`` as for :func:`paged_kv_append`. Returns the rotated q
    [T, Hq, D] bf16 (``out``, which may be q). A position outside the table gives a zero q
    row, writes no K or V and is flagged DEV_BAD_POSITION in ``status`` (int32 [1])."""
    return _rotate_append(KV_BF16, q, k, v, positions, cos_sin, k_cache, v_cache, None, None,
                          slot_mapping, q_norm, k_norm, eps, interleaved, out, status)


def paged_kv_rotate_append_q8(q, k, v, positions, cos_sin, k_cache, v_cache, k_scale, v_scale,
                              slot_mapping, fmt="e5m2", q_norm=None, k_norm=None, eps=1e-6,
                              interleaved=False, out=None, status=None):
    """:func:`paged_kv_rotate_append` into a one-byte cache: int8 codes (INT8), or FP8 codes
    (uint8 with ``fmt`` "e4m3" / "e5m2", or the matching torch float8 dtype), with
    per-(token, KV head) fp32 scales ``k_scale``/``v_scale`` [NB, Hkv, bs], quantised as
    :func:`paged_kv_append_int8` / :func:`paged_kv_append_fp8` do."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    return _rotate_append(_q8_kind(k_cache, fmt), q, k, v, positions, cos_sin, k_cache, v_cache,
                          k_scale, v_scale, slot_mapping, q_norm, k_norm, eps, interleaved, out,
                          status)


def paged_kv_gather(k_cache, v_cache, block_tables, out_offsets, num_tokens=None,
                    token_starts=None, k_scale=None, v_scale=None, fmt="e5m2", out_k=None,
                    out_v=None, status=None):
    """Cached rows read back as dense bf16 rows: row ``out_offsets[s] + i`` of the result is
    token ``token_starts[s] + i`` (0 without ``token_starts``) of sequence s.

    Caches [NB, Hkv, bs, D] bf16, or one-byte codes with ``k_scale``/``v_scale`` as for
    :func:`paged_decode_attention_multi_q8` (a value is code times scale, rounded once);
    block_tables [B, MBS] int32; out_offsets [B + 1] int32, never falling; token_starts [B]
    int32. Returns (out_k, out_v), [num_tokens, Hkv, D] bf16: the tensors given, whose rows
    past ``out_offsets[B]`` stay as they were, or new ones of ``num_tokens`` rows. A token
    outside its table row or a block id outside the pool gives a zero row, flagged in
    ``status`` (int32 [1])."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    kv = KV_BF16 if k_cache.dtype is _BF16 else _q8_kind(k_cache, fmt)
    index, (nb, hkv, bs, d) = _need_caches(kv, k_cache, v_cache, k_scale, v_scale)
    _need(block_tables, "block_tables", _I32, 2, index)
    _need(out_offsets, "out_offsets", _I32, 1, index)
    B, mbs = block_tables.shape
    _same_shape(out_offsets, "out_offsets", (B + 1,))
    if token_starts is not None:
        _need(token_starts, "token_starts", _I32, 1, index)
        _same_shape(token_starts, "token_starts", (B,))
    if num_tokens is None:
        given = out_k if out_k is not None else out_v
        if not isinstance(given, torch.Tensor):
            raise ValueError("num_tokens is needed without out_k or out_v")
        num_tokens = given.shape[0]
    rows = (num_tokens, hkv, d)
    outs = []
    for t, n in ((out_k, "out_k"), (out_v, "out_v")):
        if t is None:
            t = torch.empty(rows, dtype=_BF16, device=k_cache.device)
        else:
            _need(t, n, _BF16, 3, index)
            if t.shape != rows:
                _same_shape(t, n, rows)
        outs.append(t)
    q8 = kv != KV_BF16
    st = _run("pkv_gather_tokens", index, outs[0].data_ptr(), outs[1].data_ptr(),
              k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr() if q8 else None,
              v_scale.data_ptr() if q8 else None, block_tables.data_ptr(),
              token_starts.data_ptr() if token_starts is not None else None,
              out_offsets.data_ptr(), num_tokens, kv, _pack_dims(B, hkv, hkv, d, bs, nb, mbs),
              _status_ptr(status, index))
    if st:
        _check(st, "pkv_gather_tokens")
    return outs[0], outs[1]


def paged_kv_resize(block_tables, context_lens, target_lens, free_blocks, free_count, block_size,
                    num_tokens=None, slot_mapping=None, positions=None, token_offsets=None,
                    status=None):
    """Sequences grow and shrink from ``context_lens`` to ``target_lens`` cached tokens (both [B]
    int32, two tensors): blocks come off and go back on the stack ``free_blocks`` ([F] int32,
    the first ``free_count`` [1] int32 ids free) and in and out of ``block_tables`` [B, MBS]
    int32, where a sequence of L tokens holds the first ceil(L / block_size) entries. In place;
    ``context_lens`` becomes ``target_lens``.

    Returns (slot_mapping, positions, token_offsets) of the new tokens, as the appends take
    them: row ``token_offsets[s] + i`` is new token i of sequence s. Slots and positions are
    [num_tokens] int64, the tensors given or new ones; rows past the last new token get slot
    -1, which the appends skip. Without ``num_tokens`` and the tensors, no rows: a call that
    only shrinks. A sequence whose blocks or rows are not there, or whose lengths do not fit its
    table row, stays as it was, flagged in ``status`` (int32 [1]: DEV_NO_BLOCKS,
    DEV_BAD_CONTEXT_LEN)."""
    if not isinstance(block_tables, _Tensor):
        raise TypeError("block_tables must be a torch.Tensor")
    index = block_tables.get_device()
    if index < 0:
        _require(block_tables, "block_tables", _I32, 2)
    _need(block_tables, "block_tables", _I32, 2, index)
    _need(context_lens, "context_lens", _I32, 1, index)
    _need(target_lens, "target_lens", _I32, 1, index)
    _need(free_blocks, "free_blocks", _I32, 1, index)
    _need(free_count, "free_count", _I32, 1, index)
    B, mbs = block_tables.shape
    if context_lens.shape[0] != B or target_lens.shape[0] != B:
        raise ValueError("context_lens / target_lens must have num_seqs rows")
    if free_count.shape[0] != 1:
        raise ValueError("free_count must have one element")
    if B and context_lens.data_ptr() == target_lens.data_ptr():
        raise ValueError("context_lens and target_lens must be two tensors")
    if num_tokens is None:
        given = slot_mapping if slot_mapping is not None else positions
        num_tokens = given.shape[0] if isinstance(given, _Tensor) else 0
    rows = []
    for t, n in ((slot_mapping, "slot_mapping"), (positions, "positions")):
        if t is None:
            t = torch.empty(num_tokens, dtype=_I64, device=block_tables.device)
        else:
            _need(t, n, _I64, 1, index)
            if t.shape[0] != num_tokens:
                _same_shape(t, n, (num_tokens,))
        rows.append(t)
    if token_offsets is None:
        token_offsets = torch.empty(B + 1, dtype=_I32, device=block_tables.device)
    else:
        _need(token_offsets, "token_offsets", _I32, 1, index)
        if token_offsets.shape[0] != B + 1:
            _same_shape(token_offsets, "token_offsets", (B + 1,))
    if B == 0:
        rows[0].fill_(-1)
        rows[1].zero_()
        token_offsets.zero_()
        return rows[0], rows[1], token_offsets
    # (heads, head_dim and num_blocks are not used: any the library takes)
    st = _run("pkv_resize_sequences", index, block_tables.data_ptr(), context_lens.data_ptr(),
              target_lens.data_ptr(), free_blocks.data_ptr(), free_count.data_ptr(),
              free_blocks.shape[0], rows[0].data_ptr(), rows[1].data_ptr(),
              token_offsets.data_ptr(), num_tokens,
              _pack_dims(B, 1, 1, 64, block_size, 1, mbs), _status_ptr(status, index))
    if st:
        _check(st, "pkv_resize_sequences")
    return rows[0], rows[1], token_offsets


def paged_kv_keep(k_cache, v_cache, block_tables, base_lens, path, kept_lens=None, k_scale=None,
                  v_scale=None, status=None):
    """The kept tokens of a draft move up in the cache: cached row ``base_lens[s] + path[s, i]``
    becomes row ``base_lens[s] + i`` for i < ``kept_lens[s]`` (``path``'s width without it), K
    and V (and scales, over one-byte codes) of every head. ``path`` [B, N] int32, its used
    entries strictly rising per sequence; ``base_lens``, ``kept_lens`` [B] int32. In place,
    bit-exact. A sequence whose lengths, path or block ids do not fit stays as it was, flagged
    in ``status`` (int32 [1])."""
    kv = _move_kv(k_cache, None)
    if kv == KV_BF16:
        k_scale = v_scale = None
    index, (nb, hkv, bs, d) = _need_caches(
        KV_FP8_E4M3 if k_cache.dtype is torch.uint8 else kv, k_cache, v_cache, k_scale, v_scale)
    _need(block_tables, "block_tables", _I32, 2, index)
    _need(base_lens, "base_lens", _I32, 1, index)
    _need(path, "path", _I32, 2, index)
    B, mbs = block_tables.shape
    if base_lens.shape[0] != B or path.shape[0] != B:
        raise ValueError("base_lens / path must have num_seqs rows")
    if kept_lens is not None:
        _need(kept_lens, "kept_lens", _I32, 1, index)
        if kept_lens.shape[0] != B:
            _same_shape(kept_lens, "kept_lens", (B,))
    q8 = kv != KV_BF16
    st = _run("pkv_keep_tokens", index, k_cache.data_ptr(), v_cache.data_ptr(),
              k_scale.data_ptr() if q8 else None, v_scale.data_ptr() if q8 else None,
              block_tables.data_ptr(), base_lens.data_ptr(), path.data_ptr(),
              kept_lens.data_ptr() if kept_lens is not None else None, path.shape[1], kv,
              _pack_dims(B, hkv, hkv, d, bs, nb, mbs), _status_ptr(status, index))
    if st:
        _check(st, "pkv_keep_tokens")


def tree_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                         max_blocks_per_seq, q_len, kv_dtype=KV_BF16, device=None):
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_tree_workspace_bytes(ctypes.byref(dims), int(q_len), int(kv_dtype),
                                                    ctypes.byref(out))
    _check(st, "pkv_decode_tree_workspace_bytes")
    return int(out.value)


def _decode_tree(kv, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, tree_mask,
                 scale, tree_lens, out, workspace, status):
    index, (nb, hkv, bs, d) = _need_caches(kv, k_cache, v_cache, k_scale, v_scale)
    _need(q, "q", _BF16, 4, index)
    _need(block_tables, "block_tables", _I32, 2, index)
    _need(context_lens, "context_lens", _I32, 1, index)
    _need(tree_mask, "tree_mask", _I64, 3, index)
    shape = q.shape
    B, n, Hq, dq = shape
    if dq != d:
        raise ValueError("cache shapes disagree with q")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    if tree_mask.shape != (B, n, (n + 63) // 64):
        _same_shape(tree_mask, "tree_mask", (B, n, (n + 63) // 64))
    lens = None
    if tree_lens is not None:
        _need(tree_lens, "tree_lens", _I32, 1, index)
        if tree_lens.shape[0] != B:
            _same_shape(tree_lens, "tree_lens", (B,))
        lens = tree_lens.data_ptr()
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", _BF16, 4, index)
        if out.shape != shape:
            _same_shape(out, "out", shape)
        if B and out.data_ptr() == q.data_ptr():
            raise ValueError("out must not be q")
    dims = _pack_dims(B, Hq, hkv, d, bs, nb, block_tables.shape[1])
    status = _status_ptr(status, index)
    rows = (block_tables.data_ptr(), context_lens.data_ptr(), tree_mask.data_ptr(), lens, n,
            float(scale))

    def go(ws, ws_bytes):
        if kv == KV_BF16:
            return _run("pkv_decode_tree_bf16", index, out.data_ptr(), q.data_ptr(),
                        k_cache.data_ptr(), v_cache.data_ptr(), *rows, dims, ws.data_ptr(),
                        ws_bytes, status)
        return _run("pkv_decode_tree_q8", index, out.data_ptr(), q.data_ptr(),
                    k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                    v_scale.data_ptr(), *rows, kv, dims, ws.data_ptr(), ws_bytes, status)

    if workspace is not None:
        st = go(*_workspace(workspace, 0, q.device))
    else:
        with torch.cuda.device(index):
            need = ctypes.c_size_t(0)
            _check(_lib().pkv_decode_tree_workspace_bytes(dims, n, kv, ctypes.byref(need)),
                   "pkv_decode_tree_workspace_bytes")
        st = go(*_workspace(None, need.value, q.device))
    if st:
        _check(st, "pkv_decode_tree_bf16" if kv == KV_BF16 else "pkv_decode_tree_q8")
    return out


def paged_decode_attention_tree(q, k_cache, v_cache, block_tables, context_lens, tree_mask, scale,
                                tree_lens=None, out=None, workspace=None, status=None):
    """Attention of a tree of drafted tokens over a paged bf16 cache.

    q [B, N, Hq, D] bf16: the tree's nodes, whose K/V are the last ``tree_lens[s]`` (N without
    it; [B] int32) of the ``context_lens[s]`` cached tokens, in node order. A node sees every
    token before the nodes, and node j where bit j % 64 of ``tree_mask[s, i, j // 64]`` is set
    ([B, N, ceil(N / 64)] int64; its own bit included). Returns out [B, N, Hq, D] bf16; rows past
    ``tree_lens[s]``, and nodes that see nothing, are zeros; it must not be ``q``. ``workspace``
    (uint8, at least :func:`tree_workspace_bytes`) and ``status`` (int32 [1]) as for
    :func:`paged_decode_attention`."""
    return _decode_tree(KV_BF16, q, k_cache, v_cache, None, None, block_tables, context_lens,
                        tree_mask, scale, tree_lens, out, workspace, status)


def paged_decode_attention_tree_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                   context_lens, tree_mask, scale, fmt="e5m2", tree_lens=None,
                                   out=None, workspace=None, status=None):
    """:func:`paged_decode_attention_tree` over a one-byte cache (codes and scales as for
    :func:`paged_decode_attention_multi_q8`)."""
    return _decode_tree(_q8_kind(k_cache, fmt), q, k_cache, v_cache, k_scale, v_scale,
                        block_tables, context_lens, tree_mask, scale, tree_lens, out, workspace,
                        status)


def prompt_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, num_q_tokens,
                           num_kv_tokens, device=None):
    dims = _pack_prompt(num_seqs, num_q_heads, num_kv_heads, head_dim, num_q_tokens,
                        num_kv_tokens, 0, 0, 0, 0)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_prompt_workspace_bytes(dims, ctypes.byref(out))
    _check(st, "pkv_prompt_workspace_bytes")
    return int(out.value)


def prompt_attention(q, k, v, q_offsets, scale, kv_offsets=None, out=None, workspace=None,
                     status=None):
    """Causal attention of whole prompts packed one after the other.

    q [Tq, Hq, D], k and v [Tk, Hkv, D] bf16 (tokens at any stride, as parts of a fused
    projection's output); sequence s has rows ``q_offsets[s]`` .. ``q_offsets[s + 1] - 1`` of q
    and those of ``kv_offsets`` (``q_offsets`` without it; both [B + 1] int32) of k and v. Its
    queries are its last tokens: query i sees keys j <= nk - nq + i. Returns out [Tq, Hq, D]
    bf16: the tensor given, whose rows outside every sequence stay as they were, or a new one.
    A query without keys gets zeros. ``out`` must not overlap an input (one that begins where an
    input begins is refused). ``workspace`` (uint8, at least :func:`prompt_workspace_bytes`);
    ``status`` (int32 [1]) flags offsets that fall or leave the arrays, whose sequences are not
    computed."""
    if not isinstance(q, _Tensor):
        raise TypeError("q must be a torch.Tensor")
    index = q.get_device()
    if index < 0:
        _require(q, "q", _BF16, 3)
    q_shape, q_stride = _token_rows(q, "q", index)
    k_shape, k_stride = _token_rows(k, "k", index)
    v_shape, v_stride = _token_rows(v, "v", index)
    tq, hq, d = q_shape
    tk, hkv, dk = k_shape
    if v_shape != k_shape:
        _same_shape(v, "v", k_shape)
    if dk != d:
        raise ValueError("k and v disagree with q in head_dim")
    _need(q_offsets, "q_offsets", _I32, 1, index)
    if kv_offsets is None:
        kv_offsets = q_offsets
    elif kv_offsets is not q_offsets:
        _need(kv_offsets, "kv_offsets", _I32, 1, index)
    B = q_offsets.shape[0] - 1
    if B < 0 or kv_offsets.shape[0] != B + 1:
        raise ValueError("q_offsets / kv_offsets must have num_seqs + 1 elements")
    if out is None:
        out, out_stride = torch.empty((tq, hq, d), dtype=_BF16, device=q.device), hq * d
    else:
        out_shape, out_stride = _token_rows(out, "out", index)
        if out_shape != q_shape:
            _same_shape(out, "out", q_shape)
        if tq and out.data_ptr() in (q.data_ptr(), k.data_ptr(), v.data_ptr()):
            raise ValueError("out must not be an input")
    dims = _pack_prompt(B, hq, hkv, d, tq, tk, out_stride, q_stride, k_stride, v_stride)
    if workspace is None:
        with torch.cuda.device(index):
            need = ctypes.c_size_t(0)
            _check(_lib().pkv_prompt_workspace_bytes(dims, ctypes.byref(need)),
                   "pkv_prompt_workspace_bytes")
        workspace, ws_bytes = _workspace(None, need.value, q.device)
    else:
        workspace, ws_bytes = _workspace(workspace, 0, q.device)
    st = _run("pkv_prompt_attention_bf16", index, out.data_ptr(), q.data_ptr(), k.data_ptr(),
              v.data_ptr(), q_offsets.data_ptr(), kv_offsets.data_ptr(), float(scale), dims,
              workspace.data_ptr(), ws_bytes, _status_ptr(status, index))
    if st:
        _check(st, "pkv_prompt_attention_bf16")
    return out


def decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           num_blocks, max_blocks_per_seq, kv_dtype=KV_BF16, device=None):
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_workspace_bytes(ctypes.byref(dims), kv_dtype, ctypes.byref(out))
    _check(st, "pkv_decode_workspace_bytes")
    return int(out.value)


def _fp8_format(fmt):
    if fmt not in FP8_FORMATS:
        raise ValueError(f"fp8 format must be one of {sorted(FP8_FORMATS)}, got {fmt!r}")
    return FP8_FORMATS[fmt]


def _code_dtypes(kv):
    """Cache tensor dtypes accepted for a KV dtype code."""
    if kv == KV_BF16:
        return (torch.bfloat16,)
    if kv == KV_INT8:
        return (torch.int8,)
    return (torch.uint8, torch.float8_e4m3fn if kv == KV_FP8_E4M3 else torch.float8_e5m2)


def _require_any(t, name, dtypes, ndim, device):
    if isinstance(t, torch.Tensor) and t.dtype in dtypes[1:]:
        dtypes = (t.dtype,)
    _require(t, name, dtypes[0], ndim, device)


def _status_word(status, device):
    """The optional device status word: None, or an int32 CUDA tensor on ``device``."""
    if status is None:
        return None
    if not isinstance(status, torch.Tensor) or not status.is_cuda or status.device != device:
        raise ValueError(f"status must be an int32 CUDA tensor on {device}")
    if status.dtype != torch.int32 or status.numel() < 1 or not status.is_contiguous():
        raise TypeError("status must be a contiguous int32 tensor of at least one element")
    return status


def _workspace(workspace, need, device):
    """(tensor, size in bytes) of the decode workspace: the caller's, checked to be a
    contiguous CUDA tensor on ``device``, when it holds ``need`` bytes; else a fresh
    uint8 buffer from torch's allocator."""
    if workspace is not None:
        if (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda
                or workspace.device != device):
            raise ValueError(f"workspace must be a CUDA tensor on {device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        nbytes = workspace.numel() * workspace.element_size()
        if nbytes >= need:
            return workspace, nbytes
    ws = torch.empty(max(int(need), 256), dtype=torch.uint8, device=device)
    return ws, ws.numel()


def _decode(kv, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
            out, workspace, status):
    dev = q.device
    status = _status_word(status, dev)
    _require(q, "q", torch.bfloat16, 3, dev)
    _require_any(k_cache, "k_cache", _code_dtypes(kv), 4, dev)
    _require_any(v_cache, "v_cache", _code_dtypes(kv), 4, dev)
    if kv != KV_BF16:
        _require(k_scale, "k_scale", torch.float32, 3, dev)
        _require(v_scale, "v_scale", torch.float32, 3, dev)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError("cache shapes disagree with q")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    _cache_shapes(k_cache, v_cache, k_scale if kv != KV_BF16 else None,
                  v_scale if kv != KV_BF16 else None)
    dims = _dims(B, Hq, k_cache, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", torch.bfloat16, 3, dev)
        _same_shape(out, "out", q.shape)
    with _OnDevice(dev):
        need = ctypes.c_size_t(0)
        _check(_lib().pkv_decode_workspace_bytes(ctypes.byref(dims), kv, ctypes.byref(need)),
               "pkv_decode_workspace_bytes")
        workspace, ws_bytes = _workspace(workspace, need.value, dev)
        if kv == KV_INT8:
            name = "pkv_decode_int8"
            st = _lib().pkv_decode_int8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
                                        _ptr(context_lens), float(scale), ctypes.byref(dims),
                                        _ptr(workspace), ws_bytes, _ptr(status),
                                        _stream(dev))
        elif kv == KV_BF16:
            name = "pkv_decode_bf16"
            st = _lib().pkv_decode_bf16(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(block_tables), _ptr(context_lens), float(scale),
                                        ctypes.byref(dims), _ptr(workspace), ws_bytes,
                                        _ptr(status), _stream(dev))
        else:
            name = "pkv_decode_fp8"
            st = _lib().pkv_decode_fp8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
                                       _ptr(context_lens), float(scale), kv, ctypes.byref(dims),
                                       _ptr(workspace), ws_bytes, _ptr(status),
                                       _stream(dev))
    _check(st, name)
    return out


def paged_decode_attention(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                           workspace=None, status=None):
    """Single-token decode attention over a bf16 paged KV cache (MHA and GQA).

    q [B, Hq, D] bf16; caches [NB, Hkv, bs, D] bf16; block_tables [B, MBS] int32;
    context_lens [B] int32. Returns out [B, Hq, D] bf16. ``workspace`` (uint8, at
    least :func:`decode_workspace_bytes`) and
    ``status`` (int32 [1]) are optional.
    """
    return _decode(KV_BF16, q, k_cache, v_cache, None, None, block_tables, context_lens, scale,
                   out, workspace, status)


def paged_decode_attention_int8(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                context_lens, scale, out=None, workspace=None, status=None):
    """As :func:`paged_decode_attention` over an INT8 cache with per-(token, KV head)
    fp32 scales ``k_scale``/``v_scale`` [NB, Hkv, bs]."""
    return _decode(KV_INT8, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   scale, out, workspace, status)


def paged_decode_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                               context_lens, scale, fmt="e5m2", out=None, workspace=None,
                               status=None):
    """As :func:`paged_decode_attention` over an FP8 cache (``fmt`` "e4m3" or "e5m2";
    codes as uint8 or the matching torch float8 dtype) with per-(token, KV head) fp32
    scales ``k_scale``/``v_scale`` [NB, Hkv, bs]."""
    return _decode(_fp8_format(fmt), q, k_cache, v_cache, k_scale, v_scale, block_tables,
                   context_lens, scale, out, workspace, status)


def diff_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                         max_blocks_per_seq, kv_dtype=KV_BF16, device=None):
    """Workspace of :func:`paged_decode_attention_diff` / ``..._diff_q8``."""
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_diff_workspace_bytes(ctypes.byref(dims), int(kv_dtype),
                                                    ctypes.byref(out))
    _check(st, "pkv_decode_diff_workspace_bytes")
    return int(out.value)


def _decode_diff(kv, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, lam,
                 scale, norm_weight, eps, out_scale, out, workspace, status):
    index, (nb, hkv, bs, d) = _need_caches(kv, k_cache, v_cache, k_scale, v_scale)
    _need(q, "q", _BF16, 3, index)
    _need(block_tables, "block_tables", _I32, 2, index)
    _need(context_lens, "context_lens", _I32, 1, index)
    _need(lam, "lam", _F32, 1, index)
    B, hq, dq = q.shape
    rows, mbs = block_tables.shape
    if dq != d:
        raise ValueError("cache shapes disagree with q")
    if rows != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    if lam.shape[0] != hq // 2:
        _same_shape(lam, "lam", (hq // 2,))
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", _BF16, 1, index)
        _same_shape(norm_weight, "norm_weight", (2 * d,))
    if out is None:
        out = torch.empty((B, hq // 2, 2 * d), dtype=_BF16, device=q.device)
    else:
        _need(out, "out", _BF16, 3, index)
        if out.shape != (B, hq // 2, 2 * d):
            _same_shape(out, "out", (B, hq // 2, 2 * d))
    dims = _pack_dims(B, hq, hkv, d, bs, nb, mbs)
    name = "pkv_decode_diff_bf16" if kv == KV_BF16 else "pkv_decode_diff_q8"
    head = (out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr())
    tail = (block_tables.data_ptr(), context_lens.data_ptr(), lam.data_ptr(),
            norm_weight.data_ptr() if norm_weight is not None else None, float(eps),
            float(out_scale), float(scale))
    if kv != KV_BF16:
        head, tail = head + (k_scale.data_ptr(), v_scale.data_ptr()), tail + (kv,)
    status = _status_ptr(status, index)

    def go(ws, nbytes):
        return _run(name, index, *head, *tail, dims, ws.data_ptr(), nbytes, status)
    st = Status.ERR_WORKSPACE
    if workspace is not None:
        st = go(*_workspace(workspace, 0, q.device))
    if st == Status.ERR_WORKSPACE:  # none given, or one that is too small
        need = ctypes.c_size_t(0)
        with torch.cuda.device(index):
            _check(_lib().pkv_decode_diff_workspace_bytes(dims, kv, ctypes.byref(need)),
                   "pkv_decode_diff_workspace_bytes")
        st = go(*_workspace(workspace, need.value, q.device))
    if st:
        _check(st, name)
    return out


def paged_decode_attention_diff(q, k_cache, v_cache, block_tables, context_lens, lam, scale,
                                norm_weight=None, eps=1e-5, out_scale=1.0, out=None,
                                workspace=None, status=None):
    """Single-token differential attention over a bf16 paged KV cache: heads go in pairs
    (2j, 2j + 1); with g = Hq / Hkv, query pair j reads KV pair p = j // g and

        o[s, j] = (softmax(scale K_2p q_2j) - lam[j] softmax(scale K_2p+1 q_2j+1)) V',

    V' = [V_2p | V_2p+1], 2 D wide; with ``norm_weight`` ([2 D] bf16) o is divided by the
    root of its mean square (plus ``eps``) and multiplied by the weight; then by
    ``out_scale``. q [B, Hq, D] bf16 with Hq and Hkv even; lam [Hq / 2] fp32; caches, tables
    and lengths as for :func:`paged_decode_attention`. Returns out [B, Hq / 2, 2 D] bf16.
    ``workspace`` (uint8, at least :func:`diff_workspace_bytes`) and ``status`` (int32 [1])
    are optional."""
    return _decode_diff(KV_BF16, q, k_cache, v_cache, None, None, block_tables, context_lens, lam,
                        scale, norm_weight, eps, out_scale, out, workspace, status)


def paged_decode_attention_diff_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                   context_lens, lam, scale, fmt="e5m2", norm_weight=None,
                                   eps=1e-5, out_scale=1.0, out=None, workspace=None,
                                   status=None):
    """:func:`paged_decode_attention_diff` over a one-byte cache: int8 codes (INT8), or FP8
    codes (uint8 with ``fmt`` "e4m3" / "e5m2", or the matching torch float8 dtype), with
    per-(token, KV head) fp32 scales ``k_scale``/``v_scale`` [NB, Hkv, bs]."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    return _decode_diff(_q8_kind(k_cache, fmt), q, k_cache, v_cache, k_scale, v_scale,
                        block_tables, context_lens, lam, scale, norm_weight, eps, out_scale, out,
                        workspace, status)


def _move_kv(k_cache, kv_dtype):
    """KV dtype code of a block move: from the cache dtype, or ``kv_dtype`` (needed for
    uint8 FP8 codes, where any one-byte code gives the same move)."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    kv = _KV_OF_DTYPE.get(k_cache.dtype, -1) if kv_dtype is None else kv_dtype
    if kv is None:
        kv = KV_FP8_E5M2                      # uint8 codes: one byte + scales
    if kv == -1:
        raise TypeError(f"unsupported cache dtype {k_cache.dtype}")
    return kv


def _move_dims(k_cache):
    nb, hkv, bs, d = k_cache.shape
    return Dims(0, hkv, hkv, d, bs, nb, 1)


def _move_caches(kv, k_cache, v_cache, k_scale, v_scale):
    """Checks the device side of a block move; returns (device, bytes of one block of
    one cache, bytes of one block's scales or 0)."""
    dev = k_cache.device
    _require(k_cache, "k_cache", k_cache.dtype, 4, dev)
    _require(v_cache, "v_cache", k_cache.dtype, 4, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache differ in shape")
    nb, hkv, bs, d = k_cache.shape
    block = hkv * bs * d * k_cache.element_size()
    if kv == KV_BF16:
        return dev, block, 0
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _require(t, n, torch.float32, 3, dev)
        if tuple(t.shape) != (nb, hkv, bs):
            raise ValueError(f"{n} must be [num_blocks, num_kv_heads, block_size]")
    return dev, block, hkv * bs * 4


def _host_buffers(kv, n, block, scale_block, host_k, host_v, host_k_scale, host_v_scale):
    """Checks that the pinned host buffers of a swap hold ``n`` packed blocks (the GPU
    reads or writes them directly, so a short buffer would be overrun)."""
    bufs = [(host_k, "host_k", block), (host_v, "host_v", block)]
    if kv != KV_BF16:
        bufs += [(host_k_scale, "host_k_scale", scale_block),
                 (host_v_scale, "host_v_scale", scale_block)]
    for t, name, per_block in bufs:
        _host(t, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.numel() * t.element_size() < n * per_block:
            raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, "
                             f"{n} blocks need {n * per_block}")


def cascade_q8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                               num_blocks, max_blocks_per_seq, prefix_blocks, kv_dtype,
                               device=None):
    """Workspace of :func:`paged_decode_attention_cascade_q8` (kv_dtype KV_INT8,
    KV_FP8_E4M3 or KV_FP8_E5M2)."""
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_cascade_q8_workspace_bytes(ctypes.byref(dims), int(prefix_blocks),
                                                          int(kv_dtype), ctypes.byref(out))
    _check(st, "pkv_decode_cascade_q8_workspace_bytes")
    return int(out.value)


def paged_decode_attention_cascade_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                      context_lens, prefix_blocks, scale, fmt="e5m2", out=None,
                                      workspace=None, status=None):
    """:func:`paged_decode_attention_cascade` over a one-byte cache: int8 codes (INT8),
    or FP8 codes (uint8 with ``fmt`` "e4m3" / "e5m2", or the matching torch float8
    dtype), with per-(token, KV head) fp32 scales ``k_scale``/``v_scale`` [NB, Hkv, bs].
    Same result as :func:`paged_decode_attention_int8` / :func:`paged_decode_attention_fp8`."""
    dev = q.device
    status = _status_word(status, dev)
    kv = _q8_kind(k_cache, fmt)
    _require(q, "q", torch.bfloat16, 3, dev)
    _require_any(k_cache, "k_cache", _code_dtypes(kv), 4, dev)
    _require_any(v_cache, "v_cache", _code_dtypes(kv), 4, dev)
    _require(k_scale, "k_scale", torch.float32, 3, dev)
    _require(v_scale, "v_scale", torch.float32, 3, dev)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError("cache shapes disagree with q")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    _cache_shapes(k_cache, v_cache, k_scale, v_scale)
    dims = _dims(B, Hq, k_cache, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", torch.bfloat16, 3, dev)
        _same_shape(out, "out", q.shape)
    with _OnDevice(dev):
        need = ctypes.c_size_t(0)
        _check(_lib().pkv_decode_cascade_q8_workspace_bytes(ctypes.byref(dims),
                                                            int(prefix_blocks), kv,
                                                            ctypes.byref(need)),
               "pkv_decode_cascade_q8_workspace_bytes")
        workspace, ws_bytes = _workspace(workspace, need.value, dev)
        st = _lib().pkv_decode_cascade_q8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
                                          _ptr(context_lens), int(prefix_blocks), float(scale),
                                          kv, ctypes.byref(dims), _ptr(workspace), ws_bytes,
                                          _ptr(status), _stream(dev))
    _check(st, "pkv_decode_cascade_q8")
    return out


def copy_blocks(k_cache, v_cache, src_ids, dst_ids, k_scale=None, v_scale=None, status=None,
                kv_dtype=None):
    """Copy-on-write block copy: block dst_ids[i] := block src_ids[i] of the K/V caches
    (and their scales, for one-byte caches). ``src_ids``/``dst_ids``: device int32.
    In place, asynchronous on the current stream."""
    kv = _move_kv(k_cache, kv_dtype)
    dev, _, _ = _move_caches(kv, k_cache, v_cache, k_scale, v_scale)
    status = _status_word(status, dev)
    for t, n in ((src_ids, "src_ids"), (dst_ids, "dst_ids")):
        _require(t, n, torch.int32, 1, dev)
    if src_ids.numel() != dst_ids.numel():
        raise ValueError("src_ids and dst_ids differ in length")
    dims = _move_dims(k_cache)
    with _OnDevice(dev):
        st = _lib().pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                    _ptr(src_ids), _ptr(dst_ids), src_ids.numel(), kv,
                                    ctypes.byref(dims), _ptr(status), _stream(dev))
    _check(st, "pkv_copy_blocks")


def _host(t, name):
    if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_pinned():
        raise ValueError(f"{name} must be a pinned host tensor")
    return t


def swap_out(k_cache, v_cache, block_ids, host_k, host_v, k_scale=None, v_scale=None,
             host_k_scale=None, host_v_scale=None, status=None, kv_dtype=None):
    """Evict blocks to pinned host memory: host_k[i] := block block_ids[i] (likewise V
    and scales). Asynchronous on the current stream."""
    kv = _move_kv(k_cache, kv_dtype)
    dev, block, scale_block = _move_caches(kv, k_cache, v_cache, k_scale, v_scale)
    status = _status_word(status, dev)
    _require(block_ids, "block_ids", torch.int32, 1, dev)
    _host_buffers(kv, block_ids.numel(), block, scale_block, host_k, host_v, host_k_scale,
                  host_v_scale)
    dims = _move_dims(k_cache)
    with _OnDevice(dev):
        st = _lib().pkv_swap_out(_ptr(host_k), _ptr(host_v), _ptr(host_k_scale),
                                 _ptr(host_v_scale), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                 _ptr(v_scale), _ptr(block_ids), block_ids.numel(), kv,
                                 ctypes.byref(dims), _ptr(status), _stream(dev))
    _check(st, "pkv_swap_out")


def swap_in(k_cache, v_cache, block_ids, host_k, host_v, k_scale=None, v_scale=None,
            host_k_scale=None, host_v_scale=None, status=None, kv_dtype=None):
    """Bring evicted blocks back: block block_ids[i] := host_k[i] (likewise V and
    scales). Asynchronous on the current stream."""
    kv = _move_kv(k_cache, kv_dtype)
    dev, block, scale_block = _move_caches(kv, k_cache, v_cache, k_scale, v_scale)
    status = _status_word(status, dev)
    _require(block_ids, "block_ids", torch.int32, 1, dev)
    _host_buffers(kv, block_ids.numel(), block, scale_block, host_k, host_v, host_k_scale,
                  host_v_scale)
    dims = _move_dims(k_cache)
    with _OnDevice(dev):
        st = _lib().pkv_swap_in(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                _ptr(host_k), _ptr(host_v), _ptr(host_k_scale),
                                _ptr(host_v_scale), _ptr(block_ids), block_ids.numel(), kv,
                                ctypes.byref(dims), _ptr(status), _stream(dev))
    _check(st, "pkv_swap_in")


def multi_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_blocks_per_seq, q_len, device=None):
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_multi_workspace_bytes(ctypes.byref(dims), int(q_len),
                                                     ctypes.byref(out))
    _check(st, "pkv_decode_multi_workspace_bytes")
    return int(out.value)


def paged_decode_attention_multi(q, k_cache, v_cache, block_tables, context_lens, scale,
                                 out=None, workspace=None, status=None):
    """Attention for q_len new tokens per sequence in one call (speculative
    verification, q_len = k + 1, or a chunk of chunked prefill, q_len up to 256):
    q [B, q_len, Hq, D] bf16; the q_len newest tokens of
    every sequence are already in the bf16 caches and counted by ``context_lens``; new
    token i attends causally to positions 0 .. context_lens - q_len + i. Returns out
    [B, q_len, Hq, D] bf16."""
    dev = q.device
    status = _status_word(status, dev)
    _require(q, "q", torch.bfloat16, 4, dev)
    _require(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _require(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    B, n, Hq, D = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError("cache shapes disagree with q")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    dims = _dims(B, Hq, k_cache, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", torch.bfloat16, 4, dev)
        _same_shape(out, "out", q.shape)
    with _OnDevice(dev):
        need = ctypes.c_size_t(0)
        _check(_lib().pkv_decode_multi_workspace_bytes(ctypes.byref(dims), n,
                                                       ctypes.byref(need)),
               "pkv_decode_multi_workspace_bytes")
        workspace, ws_bytes = _workspace(workspace, need.value, dev)
        st = _lib().pkv_decode_multi_bf16(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(block_tables), _ptr(context_lens), n,
                                          float(scale), ctypes.byref(dims), _ptr(workspace),
                                          ws_bytes, _ptr(status), _stream(dev))
    _check(st, "pkv_decode_multi_bf16")
    return out


def multi_q8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                             num_blocks, max_blocks_per_seq, q_len, kv_dtype, device=None):
    """Workspace of :func:`paged_decode_attention_multi_q8` (kv_dtype KV_INT8,
    KV_FP8_E4M3 or KV_FP8_E5M2)."""
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_multi_q8_workspace_bytes(ctypes.byref(dims), int(q_len),
                                                        int(kv_dtype), ctypes.byref(out))
    _check(st, "pkv_decode_multi_q8_workspace_bytes")
    return int(out.value)


def _q8_kind(k_cache, fmt):
    """KV dtype code of a one-byte cache: int8 codes, or FP8 codes (uint8 with ``fmt``,
    or a torch float8 dtype)."""
    if k_cache.dtype == torch.int8:
        return KV_INT8
    if k_cache.dtype == torch.float8_e4m3fn:
        return KV_FP8_E4M3
    if k_cache.dtype == torch.float8_e5m2:
        return KV_FP8_E5M2
    if k_cache.dtype == torch.uint8:
        return _fp8_format(fmt)
    raise TypeError(f"a one-byte cache holds int8, uint8 or float8 codes, not {k_cache.dtype}")


def paged_decode_attention_multi_q8(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                    context_lens, scale, fmt="e5m2", out=None, workspace=None,
                                    status=None):
    """:func:`paged_decode_attention_multi` over a one-byte cache: int8 codes (INT8), or
    FP8 codes (uint8 with ``fmt`` "e4m3" / "e5m2", or the matching torch float8 dtype),
    with per-(token, KV head) fp32 scales ``k_scale``/``v_scale`` [NB, Hkv, bs]."""
    dev = q.device
    status = _status_word(status, dev)
    kv = _q8_kind(k_cache, fmt)
    _require(q, "q", torch.bfloat16, 4, dev)
    _require_any(k_cache, "k_cache", _code_dtypes(kv), 4, dev)
    _require_any(v_cache, "v_cache", _code_dtypes(kv), 4, dev)
    _require(k_scale, "k_scale", torch.float32, 3, dev)
    _require(v_scale, "v_scale", torch.float32, 3, dev)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    B, n, Hq, D = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError("cache shapes disagree with q")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    _cache_shapes(k_cache, v_cache, k_scale, v_scale)
    dims = _dims(B, Hq, k_cache, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", torch.bfloat16, 4, dev)
        _same_shape(out, "out", q.shape)
    with _OnDevice(dev):
        need = ctypes.c_size_t(0)
        _check(_lib().pkv_decode_multi_q8_workspace_bytes(ctypes.byref(dims), n, kv,
                                                          ctypes.byref(need)),
               "pkv_decode_multi_q8_workspace_bytes")
        workspace, ws_bytes = _workspace(workspace, need.value, dev)
        st = _lib().pkv_decode_multi_q8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
                                        _ptr(context_lens), n, float(scale), kv,
                                        ctypes.byref(dims), _ptr(workspace), ws_bytes,
                                        _ptr(status), _stream(dev))
    _check(st, "pkv_decode_multi_q8")
    return out


def cascade_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                            num_blocks, max_blocks_per_seq, prefix_blocks, device=None):
    dims = Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                max_blocks_per_seq)
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = _lib().pkv_decode_cascade_workspace_bytes(ctypes.byref(dims), int(prefix_blocks),
                                                       ctypes.byref(out))
    _check(st, "pkv_decode_cascade_workspace_bytes")
    return int(out.value)


def paged_decode_attention_cascade(q, k_cache, v_cache, block_tables, context_lens,
                                   prefix_blocks, scale, out=None, workspace=None, status=None):
    """Decode attention for a batch whose tables all start with the same
    ``prefix_blocks`` physical blocks (row 0's): the shared prefix is attended once
    per KV head for every query row as a dense tensor-core contraction, the suffixes by
    the ordinary decode. Same result as :func:`paged_decode_attention` (bf16 caches)."""
    dev = q.device
    status = _status_word(status, dev)
    _require(q, "q", torch.bfloat16, 3, dev)
    _require(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _require(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError("cache shapes disagree with q")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    dims = _dims(B, Hq, k_cache, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", torch.bfloat16, 3, dev)
        _same_shape(out, "out", q.shape)
    with _OnDevice(dev):
        need = ctypes.c_size_t(0)
        _check(_lib().pkv_decode_cascade_workspace_bytes(ctypes.byref(dims), int(prefix_blocks),
                                                         ctypes.byref(need)),
               "pkv_decode_cascade_workspace_bytes")
        workspace, ws_bytes = _workspace(workspace, need.value, dev)
        st = _lib().pkv_decode_cascade_bf16(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                            _ptr(block_tables), _ptr(context_lens),
                                            int(prefix_blocks), float(scale), ctypes.byref(dims),
                                            _ptr(workspace), ws_bytes, _ptr(status),
                                            _stream(dev))
    _check(st, "pkv_decode_cascade_bf16")
    return out
