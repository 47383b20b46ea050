"""Python binding of libnvfp4kv (the C ABI in include/nvfp4kv.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  There is no fallback:
if the shared library is missing or fails to load, importing the binding's
functions raises.

Functions carry the C names and take torch tensors:

  write path
    nvfp4kv_quantize_append(cache, k_new, v_new, slot_mapping, dev_status=None)
    fp8kv_quantize_append(cache, k_new, v_new, slot_mapping, dev_status=None)
  decode path
    nvfp4kv_paged_decode(cache, q, block_table, seq_lens, out, workspace, ...)
    nvfp4kv_append_paged_decode(cache, k_new, v_new, q, block_table, seq_lens, out, workspace, ...)
    nvfp4kv_paged_decode_multi(cache, q, block_table, seq_lens, out, workspace, ...)
    nvfp4kv_paged_decode_static_scratch(cache, q, block_table, seq_lens, out, ...)
    fp8kv_paged_decode / fp8kv_append_paged_decode (the FP8 comparison cache)
    nvfp4kv_decode_workspace_size(num_workers=0), new_workspace(num_workers=0)
  extend path
    nvfp4kv_dequant_prefix_fp8(cache, block_table, prefix_lens, kv_indptr, k_out, v_out)
    nvfp4kv_extend_attention_fp8(q, q_indptr, k_prefix, v_prefix, kv_indptr, prefix_lens, k_chunk, v_chunk, ...)
    nvfp4kv_extend_attention_fp8_append(cache, slot_mapping, q, q_indptr, ...)
    nvfp4kv_paged_extend(cache, q, q_indptr, block_table, seq_lens, out, workspace, ...)
    nvfp4kv_paged_extend_workspace_size(...), new_extend_workspace(...)
  around a step
    nvfp4kv_plan_step(context_lens, new_lens, block_table, num_pages, free_pages, num_free, ...)
    nvfp4kv_release_pages(old_lens, keep_lens, block_table, num_pages, free_pages, num_free, ...)
    nvfp4kv_qk_norm_rope(q, k, positions, q_out, k_out, rope=None, q_weight=None, k_weight=None, ...)
    nvfp4kv_qk_norm_rope_append(cache, q, k, v, positions, slot_mapping, q_out, rope=None, ...)
  block-scaled FP8 cache (FP8BlockCache)
    fp8bkv_append(cache, k_new, v_new, q_indptr, block_table, seq_lens, dev_status=None)
    fp8bkv_dequant(cache, block_table, lens, kv_indptr, k_out, v_out, dev_status=None)
    fp8bkv_paged_decode(cache, q, block_table, seq_lens, out, workspace, ...)
  attention over selected pages (either cache)
    nvfp4kv_page_bounds / fp8bkv_page_bounds(cache, bounds, block_table, seq_lens, from_lens=None, ...)
    nvfp4kv_select_pages(bounds, q, block_table, seq_lens, pages, first_pages=1, last_pages=1, ...)
    nvfp4kv_selected_decode / fp8bkv_selected_decode(cache, q, block_table, seq_lens, pages, out, workspace, ...)
  utilities
    nvfp4kv_read_device_status(dev_status, stream=None)
    nvfp4kv_set_wait_limit(polls) (failure detection: when bounded waits give up)
    nvfp4kv_cache_bytes / fp8kv_cache_bytes / nvfp4kv_status_string / nvfp4kv_version

``NVFP4Cache`` and ``FP8Cache`` hold the pool tensors and build the C structs;
``Rope`` holds a position rotation.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

from . import _build

PAGE_SIZE = 16
HEAD_DIM = 128

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_CHECK = 0, 1, 2, 3, 4, 5
DEV_BAD_PAGE, DEV_BAD_SLOT, DEV_BAD_LEN, DEV_TIMEOUT, DEV_NO_PAGES = 0x1, 0x2, 0x4, 0x8, 0x10
F32, BF16, E4M3 = 0, 1, 2
STATIC_SCRATCH_MAX_WORKERS = 3024   # NVFP4KV_STATIC_SCRATCH_MAX_WORKERS

_lock = threading.Lock()
_lib = None


class Nvfp4kvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


NVFP4_RECORD_BYTES = 2304      # one page-head record: K, V data and scales
FP8_RECORD_BYTES = 4096
FP8_BLOCK_RECORD_BYTES = 4128


class _Nvfp4Cache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("global_scale", ctypes.c_float), ("head_scales", ctypes.c_void_p)]


class _Fp8Cache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Fp8BlockCache(ctypes.Structure):
    _fields_ = _Fp8Cache._fields_


class _Bounds(ctypes.Structure):
    _fields_ = [("bounds", ctypes.c_void_p), ("steps", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _HeadNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int),
                ("eps", ctypes.c_float)]


_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_st = ctypes.c_int


def library_path() -> str:
    """The library that load() opens: libnvfp4kv.so built in-tree, or a prebuilt
    copy of the same sources named by NVFP4KV_LIBRARY (for example a build with
    host-side sanitizers)."""
    return os.environ.get("NVFP4KV_LIBRARY") or _build.LIB


def load(build_if_missing: bool = True):
    """Load libnvfp4kv.so (building it in-tree first if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if path == _build.LIB and not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"libnvfp4kv.so not built at {path}")
            _build.build()
        try:
            import torch  # noqa: F401  (loads the CUDA runtime torch uses first)
        except ImportError:
            pass
        lib = ctypes.CDLL(path)
        sig = {
            "nvfp4kv_quantize_append": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _vp, _st, _i32, _vp, _vp, _vp]),
            "nvfp4kv_decode_workspace_size": (ctypes.c_size_t, [_i32]),
            "nvfp4kv_paged_decode": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _i32, _i32, _vp, _i32, _vp,
                                           ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _i32, _vp, _vp]),
            "nvfp4kv_append_paged_decode": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _vp, _st, _vp, _i32, _i32,
                                                  _vp, _i32, _vp, ctypes.c_float, _vp, _st, _vp,
                                                  ctypes.c_size_t, _i32, _vp, _vp]),
            "fp8kv_append_paged_decode": (_st, [ctypes.POINTER(_Fp8Cache), _vp, _vp, _st, _vp, _i32, _i32,
                                                _vp, _i32, _vp, ctypes.c_float, _vp, _st, _vp,
                                                ctypes.c_size_t, _i32, _vp, _vp]),
            "nvfp4kv_paged_decode_multi": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _i32, _i32, _i32, _vp, _i32,
                                                 _vp, ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _i32, _vp,
                                                 _vp]),
            "nvfp4kv_paged_decode_static_scratch": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _i32, _i32, _vp,
                                                          _i32, _vp, ctypes.c_float, _vp, _st, _i32, _vp,
                                                          _vp]),
            "nvfp4kv_dequant_prefix_fp8": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _i32, _vp, _vp, _i32,
                                                 _vp, _vp, _vp, _vp]),
            "nvfp4kv_extend_attention_fp8": (_st, [_vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, ctypes.c_int64, _vp,
                                                   _vp, _st, _i32, _i32, _i32, ctypes.c_float, _vp, _st, _vp,
                                                   _vp]),
            "nvfp4kv_extend_attention_fp8_append": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _vp, _vp, _i32, _i32,
                                                          _vp, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, _st,
                                                          _i32, _i32, ctypes.c_float, _vp, _st, _vp, _vp]),
            "nvfp4kv_paged_extend": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp,
                                           _i32, ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _vp, _vp]),
            "nvfp4kv_paged_extend_workspace_size": (ctypes.c_size_t, [_i32] * 7),
            "nvfp4kv_plan_step": (_st, [_vp, _vp, _i32, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _i32, _vp, _vp]),
            "nvfp4kv_release_pages": (_st, [_vp, _vp, _i32, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp]),
            "nvfp4kv_qk_norm_rope": (_st, [_vp, _i64, _vp, _i64, _st, _i32, _i32, _i32, _vp, ctypes.POINTER(_Rope),
                                           ctypes.POINTER(_HeadNorm), _vp, _vp, _vp, _vp]),
            "nvfp4kv_qk_norm_rope_append": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _i64, _vp, _i64, _vp, _i64, _st,
                                                  _i32, _i32, _vp, _vp, ctypes.POINTER(_Rope),
                                                  ctypes.POINTER(_HeadNorm), _vp, _vp, _vp]),
            "fp8kv_quantize_append": (_st, [ctypes.POINTER(_Fp8Cache), _vp, _vp, _st, _i32, _vp, _vp, _vp]),
            "fp8kv_paged_decode": (_st, [ctypes.POINTER(_Fp8Cache), _vp, _i32, _i32, _vp, _i32, _vp,
                                         ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _i32, _vp, _vp]),
            "fp8bkv_append": (_st, [ctypes.POINTER(_Fp8BlockCache), _vp, _vp, _st, _i32, _vp, _i32, _vp, _i32, _vp, _vp,
                                    _vp]),
            "fp8bkv_dequant": (_st, [ctypes.POINTER(_Fp8BlockCache), _vp, _i32, _vp, _vp, _i32, _vp, _vp, _st, _vp, _vp]),
            "fp8bkv_paged_decode": (_st, [ctypes.POINTER(_Fp8BlockCache), _vp, _i32, _i32, _i32, _vp, _i32, _vp,
                                          ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _i32, _vp, _vp]),
            "nvfp4kv_page_bounds": (_st, [ctypes.POINTER(_Nvfp4Cache), ctypes.POINTER(_Bounds), _vp, _i32, _vp, _vp,
                                          _i32, _vp, _vp]),
            "fp8bkv_page_bounds": (_st, [ctypes.POINTER(_Fp8BlockCache), ctypes.POINTER(_Bounds), _vp, _i32, _vp, _vp,
                                         _i32, _vp, _vp]),
            "nvfp4kv_select_pages": (_st, [ctypes.POINTER(_Bounds), _vp, _i32, _i32, _i32, _vp, _i32, _vp, _i32, _i32,
                                           _i32, _vp, _vp, _vp]),
            "nvfp4kv_selected_decode": (_st, [ctypes.POINTER(_Nvfp4Cache), _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp,
                                              _i32, ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _i32, _vp, _vp]),
            "fp8bkv_selected_decode": (_st, [ctypes.POINTER(_Fp8BlockCache), _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp,
                                             _i32, ctypes.c_float, _vp, _st, _vp, ctypes.c_size_t, _i32, _vp, _vp]),
            "fp8bkv_cache_bytes": (ctypes.c_int64, [_i32, _i32, _i32, _i32]),
            "nvfp4kv_cache_bytes": (ctypes.c_int64, [_i32, _i32, _i32, _i32]),
            "fp8kv_cache_bytes": (ctypes.c_int64, [_i32, _i32, _i32, _i32]),
            "nvfp4kv_status_string": (ctypes.c_char_p, [_st]),
            "nvfp4kv_read_device_status": (_st, [_vp, _vp, ctypes.POINTER(_i32)]),
            "nvfp4kv_version": (_i32, []),
            "nvfp4kv_set_wait_limit": (ctypes.c_uint32, [ctypes.c_uint32]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(status: int, what: str) -> None:
    if status != OK:
        raise Nvfp4kvError(status, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_raw_stream = None        # torch's query of a device's current stream, once looked up (False: it has none)
_device = None            # ... of the current device


def _stream(stream, dev=None) -> int | None:
    global _raw_stream
    if stream is None:
        # the handle alone, without the Stream object around it (3 us a call)
        if _raw_stream is None:
            import torch
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", False)
        if _raw_stream and dev is not None:
            return _raw_stream(dev)
        import torch
        if _raw_stream:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_int_t = _bf16_t = _byte_t = None      # torch's types, once a call has looked the device up (torch is imported late)
_codes = {}


def _types() -> None:
    global _int_t, _bf16_t, _byte_t
    import torch
    _int_t, _bf16_t, _byte_t = torch.int32, torch.bfloat16, torch.uint8
    _codes.update({torch.float32: F32, torch.bfloat16: BF16})


def _dtype_code(t) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        _types()
        code = _codes.get(t.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
    return code


# --- caches -----------------------------------------------------------------

class NVFP4Cache:
    """An NVFP4 pool: uint8 [num_pages][num_kv_heads][NVFP4_RECORD_BYTES] page-head
    records (layout in include/nvfp4kv.h).  global_scale is the FP32 tensor
    scale G: a cached value is G * E4M3 block scale * E2M1 code.  head_scales
    (optional): per-head factors [2][num_kv_heads] (K, then V); kv head h then
    uses fl32(G * factor) as its tensor scale."""

    record_bytes = NVFP4_RECORD_BYTES

    def __init__(self, pool, global_scale: float = 1.0, head_scales=None):
        self.pool = pool
        self.num_pages, self.num_kv_heads, rb = pool.shape
        assert rb == self.record_bytes
        self.page_size, self.head_dim = PAGE_SIZE, HEAD_DIM
        self.global_scale = float(global_scale)
        self._hs = None
        if head_scales is not None:
            vals = [float(v) for row in head_scales for v in row]
            assert len(vals) == 2 * self.num_kv_heads, "head_scales: [2][num_kv_heads]"
            self._hs = (ctypes.c_float * len(vals))(*vals)     # host array the library reads per call
        self.head_scales = head_scales
        self._c = _Nvfp4Cache(pool.data_ptr(), self.num_pages, self.num_kv_heads, PAGE_SIZE, HEAD_DIM,
                              self.global_scale, None if self._hs is None else ctypes.addressof(self._hs))

    @classmethod
    def allocate(cls, num_pages, num_kv_heads, device="cuda", zero=True, **kw):
        import torch
        f = torch.zeros if zero else torch.empty
        return cls(f((num_pages, num_kv_heads, cls.record_bytes), dtype=torch.uint8, device=device), **kw)

    @property
    def c(self):
        return ctypes.byref(self._c)

    def nbytes(self) -> int:
        return self.pool.numel()


class FP8Cache(NVFP4Cache):
    """An FP8-E4M3 pool: uint8 [num_pages][num_kv_heads][FP8_RECORD_BYTES] records."""

    record_bytes = FP8_RECORD_BYTES
    _struct = _Fp8Cache

    def __init__(self, pool):
        self.pool = pool
        self.num_pages, self.num_kv_heads, rb = pool.shape
        assert rb == self.record_bytes
        self.page_size, self.head_dim = PAGE_SIZE, HEAD_DIM
        self._c = self._struct(pool.data_ptr(), self.num_pages, self.num_kv_heads, PAGE_SIZE, HEAD_DIM)


def _whole(t, name, dtype) -> None:
    """Check a tensor whose address a handle keeps: type, contiguous."""
    if str(t.dtype) != "torch." + dtype:
        raise TypeError(f"{name}: expected torch.{dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


class FP8BlockCache(FP8Cache):
    """An FP8-E4M3 pool with a scale for each page and kv head: uint8
    [num_pages][num_kv_heads][FP8_BLOCK_RECORD_BYTES] records."""

    record_bytes = FP8_BLOCK_RECORD_BYTES
    _struct = _Fp8BlockCache

    def __init__(self, pool):
        _whole(pool, "pool", "uint8")
        super().__init__(pool)
        self._span = (pool.data_ptr(), pool.data_ptr() + pool.nbytes)


class PageBounds:
    """Bounds of the keys of a cache's pages: bounds int8
    [num_pages][num_kv_heads][2][128] (least, largest), steps fp32
    [num_pages][num_kv_heads]."""

    def __init__(self, bounds, steps):
        _whole(bounds, "bounds", "int8")
        _whole(steps, "steps", "float32")
        self.num_pages, self.num_kv_heads = steps.shape
        if bounds.shape != (self.num_pages, self.num_kv_heads, 2, HEAD_DIM) or bounds.device != steps.device:
            raise ValueError(f"bounds: expected shape {(self.num_pages, self.num_kv_heads, 2, HEAD_DIM)} on "
                             f"{steps.device}, got {tuple(bounds.shape)} on {bounds.device}")
        self.bounds, self.steps = bounds, steps
        self._c = _Bounds(bounds.data_ptr(), steps.data_ptr(), self.num_pages, self.num_kv_heads)
        self.c = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, num_pages, num_kv_heads, device="cuda"):
        import torch
        return cls(torch.zeros((num_pages, num_kv_heads, 2, HEAD_DIM), dtype=torch.int8, device=device),
                   torch.zeros((num_pages, num_kv_heads), dtype=torch.float32, device=device))


class Rope:
    """A position rotation: inv_freq (rotary_dim / 2 host floats, radians a
    position; any scaling of long contexts is already in them), the pairing
    (half-split, or interleaved) and a factor on cos and sin."""

    def __init__(self, inv_freq, interleaved: bool = False, scale: float = 1.0):
        vals = [float(v) for v in inv_freq]
        self._f = (ctypes.c_double * max(1, len(vals)))(*vals)     # host array the library reads per call
        self.rotary_dim, self.interleaved, self.scale = 2 * len(vals), bool(interleaved), float(scale)
        self._c = _Rope(ctypes.addressof(self._f), self.rotary_dim, int(self.interleaved), self.scale)
        self.c = ctypes.byref(self._c)


def _current_device() -> int:
    """The current CUDA device; -1, which the checks refuse, where there is none."""
    global _device
    try:
        if _device is None:
            import torch
            _types()
            _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        return _device()
    except (AssertionError, RuntimeError):
        return -1


def _bad(t, name, dtype, shape, dev):
    """Raise for a tensor argument that is not what the call needs."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name}: not on the current CUDA device")
    raise ValueError(f"{name}: must be contiguous")


def _tensors(dev, dtype, *args) -> None:
    """Check (tensor, name, shape) arguments, None tensors passed over: type,
    shape, on device dev, contiguous."""
    for t, name, shape in args:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.get_device() == dev and
                                  t.is_contiguous()):
            _bad(t, name, dtype, shape, dev)
    if dev < 0:
        raise ValueError("no CUDA device")


def _token_rows(dev, t, name, dtype, shape) -> int:
    """Check rows [tokens][heads][128] that may be strided by token (views of a
    fused projection); returns the token stride in elements."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or dev < 0:
        _bad(t, name, dtype, shape, dev)
    step, head, one = t.stride()
    if shape[0] > 0 and (one != 1 or (shape[1] > 1 and head != shape[2])):
        raise ValueError(f"{name}: heads and channels must be contiguous")
    return step if shape[0] > 1 else shape[1] * shape[2]


def _int32(x, name) -> int:
    """An integer argument of the library's 32-bit parameters (ctypes would cut
    a larger one to its low bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


def _window(x) -> int:
    """A sliding window; one past 32 bits is longer than any sequence."""
    return _int32(min(int(x), 2 ** 31 - 1), "window")


# --- entry points -------------------------------------------------------------

def nvfp4kv_quantize_append(cache: NVFP4Cache, k_new, v_new, slot_mapping, dev_status=None,
                            stream=None) -> None:
    st = load().nvfp4kv_quantize_append(cache.c, _ptr(k_new), _ptr(v_new), _dtype_code(k_new),
                                        k_new.shape[0], _ptr(slot_mapping), _ptr(dev_status),
                                        _stream(stream))
    _check(st, "nvfp4kv_quantize_append")


def fp8kv_quantize_append(cache: FP8Cache, k_new, v_new, slot_mapping, dev_status=None,
                          stream=None) -> None:
    st = load().fp8kv_quantize_append(cache.c, _ptr(k_new), _ptr(v_new), _dtype_code(k_new),
                                      k_new.shape[0], _ptr(slot_mapping), _ptr(dev_status),
                                      _stream(stream))
    _check(st, "fp8kv_quantize_append")


def nvfp4kv_decode_workspace_size(num_workers: int = 0) -> int:
    return int(load().nvfp4kv_decode_workspace_size(int(num_workers)))


def _decode(fn, name, cache, q, block_table, seq_lens, out, workspace, sm_scale, num_workers,
            dev_status, stream):
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    B, Hq, _ = q.shape
    st = fn(cache.c, _ptr(q), B, Hq, _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
            float(sm_scale), _ptr(out), _dtype_code(out), _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            int(num_workers), _ptr(dev_status), _stream(stream))
    _check(st, name)


def nvfp4kv_paged_decode(cache: NVFP4Cache, q, block_table, seq_lens, out, workspace,
                         sm_scale=None, num_workers=0, dev_status=None, stream=None) -> None:
    _decode(load().nvfp4kv_paged_decode, "nvfp4kv_paged_decode", cache, q, block_table, seq_lens,
            out, workspace, sm_scale, num_workers, dev_status, stream)


def nvfp4kv_paged_decode_multi(cache: NVFP4Cache, q, block_table, seq_lens, out, workspace,
                               sm_scale=None, num_workers=0, dev_status=None, stream=None) -> None:
    """q: bf16 [batch][q_len][Hq][128] (the last q_len positions of each
    sequence, causal); out: [batch][q_len][Hq][128]."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    B, T, Hq, _ = q.shape
    st = load().nvfp4kv_paged_decode_multi(
        cache.c, _ptr(q), B, T, Hq, _ptr(block_table), block_table.shape[1], _ptr(seq_lens), float(sm_scale),
        _ptr(out), _dtype_code(out), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), int(num_workers),
        _ptr(dev_status), _stream(stream))
    _check(st, "nvfp4kv_paged_decode_multi")


def fp8kv_paged_decode(cache: FP8Cache, q, block_table, seq_lens, out, workspace,
                       sm_scale=None, num_workers=0, dev_status=None, stream=None) -> None:
    _decode(load().fp8kv_paged_decode, "fp8kv_paged_decode", cache, q, block_table, seq_lens,
            out, workspace, sm_scale, num_workers, dev_status, stream)


def _append_decode(fn, name, cache, k_new, v_new, q, block_table, seq_lens, out, workspace, sm_scale,
                   num_workers, dev_status, stream):
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    B, Hq, _ = q.shape
    st = fn(cache.c, _ptr(k_new), _ptr(v_new), _dtype_code(k_new), _ptr(q), B, Hq, _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), float(sm_scale), _ptr(out), _dtype_code(out),
            _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
            int(num_workers), _ptr(dev_status), _stream(stream))
    _check(st, name)


def nvfp4kv_append_paged_decode(cache: NVFP4Cache, k_new, v_new, q, block_table, seq_lens, out,
                                workspace, sm_scale=None, num_workers=0, dev_status=None,
                                stream=None) -> None:
    """One decode step: append k_new/v_new [B][Hkv][128] at position seq_lens-1, then decode."""
    _append_decode(load().nvfp4kv_append_paged_decode, "nvfp4kv_append_paged_decode", cache, k_new,
                   v_new, q, block_table, seq_lens, out, workspace, sm_scale, num_workers, dev_status,
                   stream)


def fp8kv_append_paged_decode(cache: FP8Cache, k_new, v_new, q, block_table, seq_lens, out,
                              workspace, sm_scale=None, num_workers=0, dev_status=None,
                              stream=None) -> None:
    _append_decode(load().fp8kv_append_paged_decode, "fp8kv_append_paged_decode", cache, k_new,
                   v_new, q, block_table, seq_lens, out, workspace, sm_scale, num_workers, dev_status,
                   stream)


def nvfp4kv_paged_decode_static_scratch(cache: NVFP4Cache, q, block_table, seq_lens, out,
                                        sm_scale=None, num_workers=0, dev_status=None,
                                        stream=None) -> None:
    """Decode for callers that cannot allocate device memory: the split-KV
    scratch is the library's own fixed array (see include/nvfp4kv.h)."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    B, Hq, _ = q.shape
    st = load().nvfp4kv_paged_decode_static_scratch(
        cache.c, _ptr(q), B, Hq, _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        float(sm_scale), _ptr(out), _dtype_code(out), int(num_workers), _ptr(dev_status),
        _stream(stream))
    _check(st, "nvfp4kv_paged_decode_static_scratch")


def nvfp4kv_dequant_prefix_fp8(cache: NVFP4Cache, block_table, prefix_lens, kv_indptr, k_out, v_out,
                               dev_status=None, stream=None) -> None:
    st = load().nvfp4kv_dequant_prefix_fp8(cache.c, _ptr(block_table), block_table.shape[1],
                                           _ptr(prefix_lens), _ptr(kv_indptr), prefix_lens.shape[0],
                                           _ptr(k_out), _ptr(v_out), _ptr(dev_status),
                                           _stream(stream))
    _check(st, "nvfp4kv_dequant_prefix_fp8")


def _chunk_dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return E4M3
    raise TypeError(f"unsupported chunk dtype {t.dtype}")


def nvfp4kv_extend_attention_fp8(q, q_indptr, k_prefix, v_prefix, kv_indptr, prefix_lens, k_chunk, v_chunk,
                                 out, max_q_len=None, sm_scale=None, dev_status=None, stream=None) -> None:
    """Extend attention: each chunk token attends over its sequence's FP8 prefix
    rows and the chunk up to itself.  q: bf16 [rows][Hq][128]; k_chunk, v_chunk:
    [rows][Hkv][128], bf16 or E4M3 bytes (uint8 or float8_e4m3fn: initial
    prefill on the prompt's FP8 K/V); k_prefix, v_prefix: E4M3 bytes
    [prefix rows][Hkv][128] (uint8 or float8_e4m3fn); q_indptr int32 [B+1],
    kv_indptr and prefix_lens int32 [B], all on the device; out: bf16 or fp32
    [rows][Hq][128].  max_q_len bounds every chunk length (read from q_indptr
    when None, which synchronises)."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    rows, Hq, _ = q.shape
    Hkv = k_chunk.shape[1]
    B = prefix_lens.shape[0]
    if max_q_len is None:
        max_q_len = int((q_indptr[1:] - q_indptr[:-1]).max().item()) if B > 0 else 0
    st = load().nvfp4kv_extend_attention_fp8(
        _ptr(q), _ptr(q_indptr), rows, int(max_q_len), _ptr(k_prefix), _ptr(v_prefix), _ptr(kv_indptr),
        _ptr(prefix_lens), k_prefix.shape[0], _ptr(k_chunk), _ptr(v_chunk), _chunk_dtype_code(k_chunk), B, Hq,
        Hkv, float(sm_scale), _ptr(out), _dtype_code(out), _ptr(dev_status), _stream(stream))
    _check(st, "nvfp4kv_extend_attention_fp8")


def nvfp4kv_extend_attention_fp8_append(cache: NVFP4Cache, slot_mapping, q, q_indptr, k_prefix, v_prefix,
                                        kv_indptr, prefix_lens, k_chunk, v_chunk, out, max_q_len=None,
                                        sm_scale=None, dev_status=None, stream=None) -> None:
    """nvfp4kv_extend_attention_fp8 that also writes the chunk's K/V (bf16 or
    E4M3, the values the attention reads) into the NVFP4 cache at slot_mapping
    (int32 [rows], device)."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    rows, Hq, _ = q.shape
    B = prefix_lens.shape[0]
    if max_q_len is None:
        max_q_len = int((q_indptr[1:] - q_indptr[:-1]).max().item()) if B > 0 else 0
    st = load().nvfp4kv_extend_attention_fp8_append(
        cache.c, _ptr(slot_mapping), _ptr(q), _ptr(q_indptr), rows, int(max_q_len), _ptr(k_prefix),
        _ptr(v_prefix), _ptr(kv_indptr), _ptr(prefix_lens), k_prefix.shape[0], _ptr(k_chunk), _ptr(v_chunk),
        _chunk_dtype_code(k_chunk), B, Hq, float(sm_scale), _ptr(out), _dtype_code(out), _ptr(dev_status),
        _stream(stream))
    _check(st, "nvfp4kv_extend_attention_fp8_append")


def nvfp4kv_paged_extend_workspace_size(q_rows, max_q_len, batch, num_q_heads, num_kv_heads, max_pages_per_seq,
                                        window=0) -> int:
    return int(load().nvfp4kv_paged_extend_workspace_size(
        _int32(q_rows, "q_rows"), _int32(max_q_len, "max_q_len"), _int32(batch, "batch"),
        _int32(num_q_heads, "num_q_heads"), _int32(num_kv_heads, "num_kv_heads"),
        _int32(max_pages_per_seq, "max_pages_per_seq"), _window(window)))


def nvfp4kv_paged_extend(cache: NVFP4Cache, q, q_indptr, block_table, seq_lens, out, workspace, max_q_len=None, window=0,
                         sm_scale=None, dev_status=None, stream=None) -> None:
    """Causal attention of a ragged chunk of tokens, already in the cache as the
    last tokens of their sequences, over the paged NVFP4 cache.  q: bf16
    [rows][Hq][128]; q_indptr int32 [B+1]; block_table int32 [B][pages];
    seq_lens int32 [B]; out: bf16 or fp32 [rows][Hq][128]; workspace: see
    new_extend_workspace (None where no bytes are needed).  max_q_len bounds
    every chunk (read from q_indptr when None, which synchronises); window 0 or
    the keys a query sees at most."""
    import torch
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    dev = _current_device()
    B, pages = block_table.shape
    rows, Hq, _ = q.shape
    _tensors(dev, torch.bfloat16, (q, "q", (rows, Hq, HEAD_DIM)))
    _tensors(dev, out.dtype, (out, "out", (rows, Hq, HEAD_DIM)))
    _tensors(dev, torch.uint8, (cache.pool, "cache", cache.pool.shape),
             (workspace, "workspace", (0 if workspace is None else workspace.numel(),)))
    _tensors(dev, torch.int32, (q_indptr, "q_indptr", (B + 1,)), (block_table, "block_table", (B, pages)),
             (seq_lens, "seq_lens", (B,)), (dev_status, "dev_status", (1,)))
    if max_q_len is None:
        max_q_len = int((q_indptr[1:] - q_indptr[:-1]).max().item()) if B > 0 else 0
    st = load().nvfp4kv_paged_extend(
        cache.c, _ptr(q), _ptr(q_indptr), rows, _int32(max_q_len, "max_q_len"), B, Hq, _ptr(block_table), pages,
        _ptr(seq_lens), _window(window), float(sm_scale), _ptr(out), _dtype_code(out), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(dev_status), _stream(stream, dev))
    _check(st, "nvfp4kv_paged_extend")


def nvfp4kv_plan_step(context_lens, new_lens, block_table, num_pages, free_pages, num_free, num_free_out, seq_lens,
                      q_indptr, slot_mapping, positions=None, kv_indptr=None, dev_status=None, stream=None) -> None:
    """A step's tables from its requests' lengths (all int32 on the device):
    takes fresh pages from the stack free_pages[: num_free], enters them into
    block_table [B][max_pages], and writes seq_lens [B], q_indptr [B+1],
    kv_indptr [B], slot_mapping and positions [max_tokens] (-1 behind the last
    token) and num_free_out [1] (which may be num_free)."""
    import torch
    dev = _current_device()
    B, pages = block_table.shape
    T, F = slot_mapping.numel(), free_pages.numel()
    _tensors(dev, torch.int32, (context_lens, "context_lens", (B,)), (new_lens, "new_lens", (B,)),
             (block_table, "block_table", (B, pages)), (free_pages, "free_pages", (F,)), (num_free, "num_free", (1,)),
             (num_free_out, "num_free_out", (1,)), (seq_lens, "seq_lens", (B,)), (q_indptr, "q_indptr", (B + 1,)),
             (slot_mapping, "slot_mapping", (T,)), (positions, "positions", (T,)), (kv_indptr, "kv_indptr", (B,)),
             (dev_status, "dev_status", (1,)))
    st = load().nvfp4kv_plan_step(
        _ptr(context_lens), _ptr(new_lens), B, _ptr(block_table), pages, _int32(num_pages, "num_pages"),
        _ptr(free_pages), F,
        _ptr(num_free), _ptr(num_free_out), _ptr(seq_lens), _ptr(q_indptr), _ptr(kv_indptr), _ptr(slot_mapping),
        _ptr(positions), T, _ptr(dev_status), _stream(stream, dev))
    _check(st, "nvfp4kv_plan_step")


def nvfp4kv_release_pages(old_lens, keep_lens, block_table, num_pages, free_pages, num_free, num_free_out,
                          dev_status=None, stream=None) -> None:
    """Put the pages that requests no longer need (old_lens down to keep_lens
    tokens, int32 [B]) back on the stack free_pages[: num_free]; num_free_out
    [1] may be num_free."""
    import torch
    dev = _current_device()
    B, pages = block_table.shape
    F = free_pages.numel()
    _tensors(dev, torch.int32, (old_lens, "old_lens", (B,)), (keep_lens, "keep_lens", (B,)),
             (block_table, "block_table", (B, pages)), (free_pages, "free_pages", (F,)), (num_free, "num_free", (1,)),
             (num_free_out, "num_free_out", (1,)), (dev_status, "dev_status", (1,)))
    st = load().nvfp4kv_release_pages(
        _ptr(old_lens), _ptr(keep_lens), B, _ptr(block_table), pages, _int32(num_pages, "num_pages"),
        _ptr(free_pages), F,
        _ptr(num_free), _ptr(num_free_out), _ptr(dev_status), _stream(stream, dev))
    _check(st, "nvfp4kv_release_pages")


def _head_norm(dev, q_weight, k_weight, eps):
    first = k_weight if q_weight is None else q_weight
    if first is None:
        return None
    _tensors(dev, first.dtype, (q_weight, "q_weight", (HEAD_DIM,)), (k_weight, "k_weight", (HEAD_DIM,)))
    return ctypes.byref(_HeadNorm(_ptr(q_weight), _ptr(k_weight), _dtype_code(first), float(eps)))


def nvfp4kv_qk_norm_rope(q, k, positions, q_out, k_out, rope: Rope | None = None, q_weight=None, k_weight=None,
                         eps=1e-6, dev_status=None, stream=None) -> None:
    """Norm (where a weight is given) and rotate each head of q [T][Hq][128] and
    k [T][Hkv][128] (fp32 or bf16; tokens may be strided, as views of a fused
    projection are) at positions int32 [T] (negative: token left out) into
    q_out (bf16) and k_out (k's type)."""
    import torch
    dev = _current_device()
    T, Hq, _ = q.shape
    Hkv, code = k.shape[1], _dtype_code(q)
    q_step = _token_rows(dev, q, "q", q.dtype, (T, Hq, HEAD_DIM))
    k_step = _token_rows(dev, k, "k", q.dtype, (T, Hkv, HEAD_DIM))
    _tensors(dev, torch.int32, (positions, "positions", (T,)), (dev_status, "dev_status", (1,)))
    _tensors(dev, torch.bfloat16, (q_out, "q_out", (T, Hq, HEAD_DIM)))
    _tensors(dev, q.dtype, (k_out, "k_out", (T, Hkv, HEAD_DIM)))
    st = load().nvfp4kv_qk_norm_rope(
        _ptr(q), q_step, _ptr(k), k_step, code, T, Hq, Hkv, _ptr(positions), None if rope is None else rope.c,
        _head_norm(dev, q_weight, k_weight, eps), _ptr(q_out), _ptr(k_out), _ptr(dev_status),
        _stream(stream, dev))
    _check(st, "nvfp4kv_qk_norm_rope")


def nvfp4kv_qk_norm_rope_append(cache: NVFP4Cache, q, k, v, positions, slot_mapping, q_out,
                                rope: Rope | None = None, q_weight=None, k_weight=None, eps=1e-6, dev_status=None,
                                stream=None) -> None:
    """nvfp4kv_qk_norm_rope with the finished keys and the values v [T][Hkv][128]
    written into the NVFP4 cache at slot_mapping int32 [T] instead of k_out."""
    import torch
    dev = _current_device()
    T, Hq, _ = q.shape
    Hkv, code = cache.num_kv_heads, _dtype_code(q)
    q_step = _token_rows(dev, q, "q", q.dtype, (T, Hq, HEAD_DIM))
    k_step = _token_rows(dev, k, "k", q.dtype, (T, Hkv, HEAD_DIM))
    v_step = _token_rows(dev, v, "v", q.dtype, (T, Hkv, HEAD_DIM))
    _tensors(dev, torch.int32, (positions, "positions", (T,)), (slot_mapping, "slot_mapping", (T,)),
             (dev_status, "dev_status", (1,)))
    _tensors(dev, torch.bfloat16, (q_out, "q_out", (T, Hq, HEAD_DIM)))
    _tensors(dev, torch.uint8, (cache.pool, "cache", cache.pool.shape))
    st = load().nvfp4kv_qk_norm_rope_append(
        cache.c, _ptr(q), q_step, _ptr(k), k_step, _ptr(v), v_step, code, T, Hq, _ptr(positions), _ptr(slot_mapping),
        None if rope is None else rope.c, _head_norm(dev, q_weight, k_weight, eps), _ptr(q_out), _ptr(dev_status),
        _stream(stream, dev))
    _check(st, "nvfp4kv_qk_norm_rope_append")


def _kind(cache, kind, dev) -> None:
    """Check a cache argument: of its kind (another one's records would be
    misread), on device dev.  (Its pool was checked as it was made.)"""
    if type(cache).record_bytes != kind.record_bytes:
        raise TypeError(f"cache: expected {kind.__name__}, got {type(cache).__name__}")
    if cache.pool.get_device() != dev or dev < 0:
        raise ValueError("cache: not on the current CUDA device")
    if not cache.pool.is_contiguous():
        raise ValueError("cache: must be contiguous")


# The calls below check each tensor in one expression of the caller's (the host's
# time is most of a short call's); what fails goes through _tensors, which says why.

def fp8bkv_append(cache: FP8BlockCache, k_new, v_new, q_indptr, block_table, seq_lens, dev_status=None,
                  stream=None) -> None:
    """Write the rows k_new, v_new [T][Hkv][128] (fp32 or bf16), sequence b's being
    q_indptr[b] .. q_indptr[b+1] - 1 (int32 [B+1]), as the last tokens of its
    seq_lens[b] (int32 [B], they included) into the pages of block_table int32
    [B][pages]; a page's scale rises where they need it."""
    dev = _current_device()
    i32 = _int_t
    _kind(cache, FP8BlockCache, dev)
    B, pages = block_table.shape
    T, code, dtype = k_new.shape[0], _dtype_code(k_new), k_new.dtype
    rows = (T, cache.num_kv_heads, HEAD_DIM)
    if not (k_new.shape == rows and k_new.get_device() == dev and k_new.is_contiguous() and
            v_new.dtype is dtype and v_new.shape == rows and v_new.get_device() == dev and v_new.is_contiguous()):
        _tensors(dev, dtype, (k_new, "k_new", rows), (v_new, "v_new", rows))
    if not (q_indptr.dtype is i32 and q_indptr.shape == (B + 1,) and q_indptr.get_device() == dev and
            q_indptr.is_contiguous() and
            block_table.dtype is i32 and block_table.get_device() == dev and block_table.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.shape == (B,) and seq_lens.get_device() == dev and
            seq_lens.is_contiguous()):
        _tensors(dev, i32, (q_indptr, "q_indptr", (B + 1,)), (block_table, "block_table", (B, pages)),
                 (seq_lens, "seq_lens", (B,)))
    if not (dev_status is None or (dev_status.dtype is i32 and dev_status.shape == (1,) and
                                   dev_status.get_device() == dev)):
        _tensors(dev, i32, (dev_status, "dev_status", (1,)))
    st = load().fp8bkv_append(cache.c, k_new.data_ptr(), v_new.data_ptr(), code, T, q_indptr.data_ptr(), B,
                              block_table.data_ptr(), pages, seq_lens.data_ptr(), _ptr(dev_status), _stream(stream, dev))
    if st:
        _check(st, "fp8bkv_append")


_HEAD_BYTES = {F32: 4 * HEAD_DIM, BF16: 2 * HEAD_DIM, E4M3: HEAD_DIM}


def fp8bkv_dequant(cache: FP8BlockCache, block_table, lens, kv_indptr, k_out, v_out, dev_status=None,
                   stream=None) -> None:
    """Read the first lens[b] cached rows of each sequence back into rows
    kv_indptr[b] .. of k_out and v_out [rows][Hkv][128]: fp32, bf16, or E4M3 at
    scale 1.0 (uint8 or float8_e4m3fn: the workspace of the extend calls, where
    values past 448 saturate and small ones lose bits)."""
    dev = _current_device()
    i32, dtype = _int_t, k_out.dtype
    _kind(cache, FP8BlockCache, dev)
    B, pages = block_table.shape
    code = _codes.get(dtype)
    if code is None:
        code = _chunk_dtype_code(k_out)
    rows = (k_out.shape[0], cache.num_kv_heads, HEAD_DIM)
    if not (k_out.shape == rows and k_out.get_device() == dev and k_out.is_contiguous() and
            v_out.dtype is dtype and v_out.shape == rows and v_out.get_device() == dev and v_out.is_contiguous()):
        _tensors(dev, dtype, (k_out, "k_out", rows), (v_out, "v_out", rows))
    if not (kv_indptr.dtype is i32 and kv_indptr.shape == (B,) and kv_indptr.get_device() == dev and
            kv_indptr.is_contiguous() and
            block_table.dtype is i32 and block_table.get_device() == dev and block_table.is_contiguous() and
            lens.dtype is i32 and lens.shape == (B,) and lens.get_device() == dev and lens.is_contiguous()):
        _tensors(dev, i32, (kv_indptr, "kv_indptr", (B,)), (block_table, "block_table", (B, pages)),
                 (lens, "lens", (B,)))
    if not (dev_status is None or (dev_status.dtype is i32 and dev_status.shape == (1,) and
                                   dev_status.get_device() == dev)):
        _tensors(dev, i32, (dev_status, "dev_status", (1,)))
    # (the call sees one row of the outputs, whose number only the device knows)
    k_at, v_at, size = k_out.data_ptr(), v_out.data_ptr(), rows[0] * rows[1] * _HEAD_BYTES[code]
    begin, end = cache._span
    if -size < k_at - v_at < size or begin - size < k_at < end or begin - size < v_at < end:
        raise ValueError("k_out, v_out: overlap one another or the cache")
    st = load().fp8bkv_dequant(cache.c, block_table.data_ptr(), pages, lens.data_ptr(), kv_indptr.data_ptr(), B,
                               k_at, v_at, code, _ptr(dev_status), _stream(stream, dev))
    if st:
        _check(st, "fp8bkv_dequant")


def _attention_tensors(dev, B, max_pages, q, block_table, seq_lens, out, workspace, dev_status):
    """Check what the decode calls share: q bf16 [B][Hq][128] or
    [B][q_len][Hq][128], out of its shape (None: there is none); returns (q_len,
    Hq, bytes of workspace)."""
    i32 = _int_t
    shape = q.shape
    q_len, heads = (1, shape[1]) if len(shape) == 3 else ((shape[1], shape[2]) if len(shape) == 4 else (-1, 0))
    if q_len < 0 or shape[0] != B or shape[-1] != HEAD_DIM:
        raise ValueError(f"q: expected [{B}][Hq][{HEAD_DIM}] or [{B}][q_len][Hq][{HEAD_DIM}], got shape {tuple(shape)}")
    if not (q.dtype is _bf16_t and q.get_device() == dev and q.is_contiguous()):
        _tensors(dev, _bf16_t, (q, "q", shape))
    if out is not None and not (out.shape == shape and out.get_device() == dev and out.is_contiguous()):
        _tensors(dev, out.dtype, (out, "out", shape))
    if not (block_table.dtype is i32 and block_table.get_device() == dev and block_table.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.shape == (B,) and seq_lens.get_device() == dev and
            seq_lens.is_contiguous()):
        _tensors(dev, i32, (block_table, "block_table", (B, max_pages)), (seq_lens, "seq_lens", (B,)))
    if not (dev_status is None or (dev_status.dtype is i32 and dev_status.shape == (1,) and
                                   dev_status.get_device() == dev)):
        _tensors(dev, i32, (dev_status, "dev_status", (1,)))
    if workspace is None:
        return q_len, heads, 0
    n = workspace.numel()
    if not (workspace.dtype is _byte_t and workspace.get_device() == dev and workspace.is_contiguous()):
        _tensors(dev, _byte_t, (workspace, "workspace", (n,)))
    return q_len, heads, n


def fp8bkv_paged_decode(cache: FP8BlockCache, q, block_table, seq_lens, out, workspace, sm_scale=None, num_workers=0,
                        dev_status=None, stream=None) -> None:
    """Decode attention over the block-scaled FP8 cache.  q: bf16 [B][Hq][128], or
    [B][q_len][Hq][128] for the last q_len positions of each sequence, causal
    among themselves; out: bf16 or fp32 of q's shape; workspace: new_workspace."""
    dev = _current_device()
    _kind(cache, FP8BlockCache, dev)
    B, pages = block_table.shape
    q_len, heads, n = _attention_tensors(dev, B, pages, q, block_table, seq_lens, out, workspace, dev_status)
    st = load().fp8bkv_paged_decode(
        cache.c, q.data_ptr(), B, q_len, heads, block_table.data_ptr(), pages, seq_lens.data_ptr(),
        _SM_SCALE if sm_scale is None else float(sm_scale), out.data_ptr(), _dtype_code(out), _ptr(workspace), n,
        _int32(num_workers, "num_workers"), _ptr(dev_status), _stream(stream, dev))
    if st:
        _check(st, "fp8bkv_paged_decode")


_SM_SCALE = 1.0 / math.sqrt(HEAD_DIM)


def _page_bounds(name, kind, cache, bounds, block_table, seq_lens, from_lens, dev_status, stream):
    dev = _current_device()
    i32 = _int_t
    _kind(cache, kind, dev)
    B, pages = block_table.shape
    if bounds.steps.get_device() != dev:
        raise ValueError("bounds: not on the current CUDA device")
    if not (block_table.dtype is i32 and block_table.get_device() == dev and block_table.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.shape == (B,) and seq_lens.get_device() == dev and
            seq_lens.is_contiguous()):
        _tensors(dev, i32, (block_table, "block_table", (B, pages)), (seq_lens, "seq_lens", (B,)))
    if not ((from_lens is None or (from_lens.dtype is i32 and from_lens.shape == (B,) and
                                   from_lens.get_device() == dev and from_lens.is_contiguous())) and
            (dev_status is None or (dev_status.dtype is i32 and dev_status.shape == (1,) and
                                    dev_status.get_device() == dev))):
        _tensors(dev, i32, (from_lens, "from_lens", (B,)), (dev_status, "dev_status", (1,)))
    st = getattr(load(), name)(cache.c, bounds.c, block_table.data_ptr(), pages, _ptr(from_lens), seq_lens.data_ptr(), B,
                               _ptr(dev_status), _stream(stream, dev))
    if st:
        _check(st, name)


def nvfp4kv_page_bounds(cache: NVFP4Cache, bounds: PageBounds, block_table, seq_lens, from_lens=None, dev_status=None,
                        stream=None) -> None:
    """Bring the bounds of the pages that tokens from_lens[b] .. seq_lens[b] - 1
    (int32 [B]; None: from 0) were written into up to date."""
    _page_bounds("nvfp4kv_page_bounds", NVFP4Cache, cache, bounds, block_table, seq_lens, from_lens, dev_status, stream)


def fp8bkv_page_bounds(cache: FP8BlockCache, bounds: PageBounds, block_table, seq_lens, from_lens=None,
                       dev_status=None, stream=None) -> None:
    """nvfp4kv_page_bounds of a block-scaled FP8 cache."""
    _page_bounds("fp8bkv_page_bounds", FP8BlockCache, cache, bounds, block_table, seq_lens, from_lens, dev_status, stream)


def _page_lists(dev, pages, B, q_len, heads, flat) -> int:
    """Check lists of pages int32 [B][q_len][Hkv][budget] (flat: or
    [B][Hkv][budget]); returns the budget."""
    shape = pages.shape
    budget = shape[-1]
    if not (pages.dtype is _int_t and pages.get_device() == dev and pages.is_contiguous() and
            (shape == (B, q_len, heads, budget) or (flat and shape == (B, heads, budget)))):
        _tensors(dev, _int_t, (pages, "pages", (B, heads, budget) if flat and len(shape) == 3
                                    else (B, q_len, heads, budget)))
    return budget


def nvfp4kv_select_pages(bounds: PageBounds, q, block_table, seq_lens, pages, first_pages=1, last_pages=1,
                         dev_status=None, stream=None) -> None:
    """Select pages for each query token and kv head: the first first_pages and
    the last last_pages that the token sees and the best of the others by the
    score of their bounds, into pages int32 [B][q_len][Hkv][budget] (ascending
    places in the sequence, -1 behind the last; [B][Hkv][budget] where q is
    [B][Hq][128])."""
    dev = _current_device()
    B, max_pages = block_table.shape
    if bounds.steps.get_device() != dev or dev < 0:
        raise ValueError("bounds: not on the current CUDA device")
    q_len, heads, _ = _attention_tensors(dev, B, max_pages, q, block_table, seq_lens, None, None, dev_status)
    budget = _page_lists(dev, pages, B, q_len, bounds.num_kv_heads, q.dim() == 3)
    st = load().nvfp4kv_select_pages(
        bounds.c, q.data_ptr(), B, q_len, heads, block_table.data_ptr(), max_pages, seq_lens.data_ptr(), budget,
        _int32(first_pages, "first_pages"), _int32(last_pages, "last_pages"), pages.data_ptr(), _ptr(dev_status),
        _stream(stream, dev))
    if st:
        _check(st, "nvfp4kv_select_pages")


def _selected_decode(name, kind, cache, q, block_table, seq_lens, pages, out, workspace, sm_scale, num_workers,
                     dev_status, stream):
    dev = _current_device()
    _kind(cache, kind, dev)
    B, max_pages = block_table.shape
    q_len, heads, n = _attention_tensors(dev, B, max_pages, q, block_table, seq_lens, out, workspace, dev_status)
    budget = _page_lists(dev, pages, B, q_len, cache.num_kv_heads, q.dim() == 3)
    st = getattr(load(), name)(
        cache.c, q.data_ptr(), B, q_len, heads, block_table.data_ptr(), max_pages, seq_lens.data_ptr(), pages.data_ptr(),
        budget, _SM_SCALE if sm_scale is None else float(sm_scale), out.data_ptr(), _dtype_code(out), _ptr(workspace), n,
        _int32(num_workers, "num_workers"), _ptr(dev_status), _stream(stream, dev))
    if st:
        _check(st, name)


def nvfp4kv_selected_decode(cache: NVFP4Cache, q, block_table, seq_lens, pages, out, workspace, sm_scale=None,
                            num_workers=0, dev_status=None, stream=None) -> None:
    """Decode attention of each query token and kv head over the pages listed for
    it (as nvfp4kv_select_pages writes them).  q, out and workspace as for
    fp8bkv_paged_decode."""
    _selected_decode("nvfp4kv_selected_decode", NVFP4Cache, cache, q, block_table, seq_lens, pages, out, workspace,
                     sm_scale, num_workers, dev_status, stream)


def fp8bkv_selected_decode(cache: FP8BlockCache, q, block_table, seq_lens, pages, out, workspace, sm_scale=None,
                           num_workers=0, dev_status=None, stream=None) -> None:
    """nvfp4kv_selected_decode over a block-scaled FP8 cache."""
    _selected_decode("fp8bkv_selected_decode", FP8BlockCache, cache, q, block_table, seq_lens, pages, out, workspace,
                     sm_scale, num_workers, dev_status, stream)


def fp8bkv_cache_bytes(num_pages, num_kv_heads, page_size=PAGE_SIZE, head_dim=HEAD_DIM) -> int:
    return int(load().fp8bkv_cache_bytes(num_pages, num_kv_heads, page_size, head_dim))


def nvfp4kv_cache_bytes(num_pages, num_kv_heads, page_size=PAGE_SIZE, head_dim=HEAD_DIM) -> int:
    return int(load().nvfp4kv_cache_bytes(num_pages, num_kv_heads, page_size, head_dim))


def fp8kv_cache_bytes(num_pages, num_kv_heads, page_size=PAGE_SIZE, head_dim=HEAD_DIM) -> int:
    return int(load().fp8kv_cache_bytes(num_pages, num_kv_heads, page_size, head_dim))


def read_device_status(dev_status, stream=None) -> int:
    """Synchronise `stream` and return the bits of the device status word
    (int32 tensor of one element); 0 when no kernel reported anything."""
    bits = _i32(0)
    st = load().nvfp4kv_read_device_status(_ptr(dev_status), _stream(stream), ctypes.byref(bits))
    if st not in (OK, ERR_DEVICE_CHECK):
        _check(st, "nvfp4kv_read_device_status")
    return int(bits.value)


nvfp4kv_read_device_status = read_device_status


def status_string(status: int) -> str:
    return load().nvfp4kv_status_string(int(status)).decode()


nvfp4kv_status_string = status_string


def nvfp4kv_version() -> int:
    return int(load().nvfp4kv_version())


WAIT_LIMIT_DEFAULT = 4194304        # NVFP4KV_WAIT_LIMIT_DEFAULT


def nvfp4kv_set_wait_limit(polls: int) -> int:
    """Polls after which a kernel's bounded waits give up (and report
    DEV_TIMEOUT), for the calls made from now on; returns the previous value."""
    return int(load().nvfp4kv_set_wait_limit(int(polls)))


def new_workspace(num_workers: int = 0, device="cuda"):
    """A decode workspace tensor of the size the library asks for."""
    import torch
    n = nvfp4kv_decode_workspace_size(num_workers)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def new_extend_workspace(q_rows, max_q_len, batch, num_q_heads, num_kv_heads, max_pages_per_seq, window=0,
                         device="cuda"):
    """A workspace tensor for nvfp4kv_paged_extend calls of these sizes."""
    import torch
    n = nvfp4kv_paged_extend_workspace_size(q_rows, max_q_len, batch, num_q_heads, num_kv_heads, max_pages_per_seq,
                                            window)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)

