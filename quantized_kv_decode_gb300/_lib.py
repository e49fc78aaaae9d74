"""ctypes binding of libkvq.so (include/kvq.h).

Argument marshalling only: every step of the work runs in the CUDA kernels of
the shared library.  If the library has not been built, every entry point
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import (POINTER, Structure, byref, c_double, c_float, c_int32, c_int64, c_size_t, c_uint8,  # noqa: F401
                    c_uint32, c_uint64, c_void_p)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

# kvq_status
KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_WORKSPACE = 3
KVQ_ERR_CUDA = 4

# bits of the device status word
KVQ_FLAG_SEQ_LEN = 0x1
KVQ_FLAG_BLOCK_TABLE = 0x2
KVQ_FLAG_ZERO_CLAMPED = 0x4
KVQ_FLAG_NONFINITE = 0x8
KVQ_FLAG_OOB = 0x10  # debug builds only: an access outside its array was skipped
KVQ_FLAG_POOL_EMPTY = 0x20
KVQ_FLAG_PAGE_LIST = 0x40
KVQ_FLAG_TIMEOUT = 0x80  # a bounded wait inside a kernel ran out

# kvq_rope_scaling
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
KVQ_ROPE_MAX_PAIRS = 128
KVQ_ROPE_MAX_AXES = 4
KVQ_MAX_POOL_BATCH = 16384
KVQ_MAX_PREFIXES = 65535

# kvq_debug_wait: the waits a debug build can let run out
(KVQ_WAIT_NONE, KVQ_WAIT_SOFTMAX, KVQ_WAIT_K, KVQ_WAIT_V, KVQ_WAIT_LOAD_K, KVQ_WAIT_LOAD_V,
 KVQ_WAIT_SCORES, KVQ_WAIT_SUM, KVQ_WAIT_COUNT) = range(9)

# kvq_array: the caller arrays a debug build checks
(KVQ_ARRAY_K_CODES, KVQ_ARRAY_V_CODES, KVQ_ARRAY_K_SCALE, KVQ_ARRAY_K_ZERO, KVQ_ARRAY_V_SCALE,
 KVQ_ARRAY_V_ZERO, KVQ_ARRAY_K_WINDOW, KVQ_ARRAY_V_WINDOW, KVQ_ARRAY_BLOCK_TABLE, KVQ_ARRAY_Q,
 KVQ_ARRAY_K_NEW, KVQ_ARRAY_V_NEW, KVQ_ARRAY_SEQ_LENS, KVQ_ARRAY_OUT,
 KVQ_ARRAY_WORKSPACE) = range(15)

KVQ_DENSE = 0
KVQ_PAGED = 1


class kvq_cache_desc(Structure):
    _fields_ = [
        ("bits", c_int32),
        ("group_size", c_int32),
        ("num_kv_heads", c_int32),
        ("head_dim", c_int32),
        ("layout", c_int32),
        ("capacity", c_int32),
        ("num_pages", c_int32),
        ("max_blocks_per_seq", c_int32),
        ("symmetric", c_int32),
        ("k_per_channel", c_int32),
        ("sink_tokens", c_int32),
        ("nf4", c_int32),
    ]


class kvq_cache(Structure):
    _fields_ = [
        ("k_codes", c_void_p),
        ("v_codes", c_void_p),
        ("k_scale", c_void_p),
        ("k_zero", c_void_p),
        ("v_scale", c_void_p),
        ("v_zero", c_void_p),
        ("block_table", c_void_p),
        ("k_window", c_void_p),
        ("v_window", c_void_p),
    ]


class kvq_rope_desc(Structure):
    _fields_ = [
        ("rotary_dim", c_int32),
        ("interleaved", c_int32),
        ("scaling", c_int32),
        ("original_context", c_int32),
        ("base", c_double),
        ("factor", c_double),
        ("low_turns", c_double),
        ("high_turns", c_double),
        ("amplitude", c_double),
    ]


class kvq_rope(Structure):
    _fields_ = [
        ("rotary_dim", c_int32),
        ("interleaved", c_int32),
        ("amplitude", c_uint64),
        ("turns", c_uint64 * KVQ_ROPE_MAX_PAIRS),
    ]


class kvq_rope_axes_desc(Structure):
    _fields_ = [
        ("rope", kvq_rope_desc),
        ("num_axes", c_int32),
        ("pairs", c_int32 * KVQ_ROPE_MAX_AXES),
        ("cycled", c_int32),
        ("own_ladders", c_int32),
    ]


class kvq_rope_axes(Structure):
    _fields_ = [
        ("rope", kvq_rope),
        ("num_axes", c_int32),
        ("axis", c_uint8 * KVQ_ROPE_MAX_PAIRS),
    ]


class kvq_page_pool(Structure):
    _fields_ = [
        ("num_pages", c_int32),
        ("page_size", c_int32),
        ("batch", c_int32),
        ("max_blocks_per_seq", c_int32),
        ("ref_count", c_void_p),
        ("block_table", c_void_p),
    ]


class KVQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_lib = None

# name -> (restype, argtypes): the C declarations of include/kvq.h
SIGNATURES = {
    "kvq_cache_bytes": (c_size_t, [POINTER(kvq_cache_desc), c_int64]),
    "kvq_cache_window_bytes": (c_size_t, [POINTER(kvq_cache_desc), c_int32]),
    "kvq_cache_array_bytes": (c_int32, [POINTER(kvq_cache_desc), c_int32,
                                        POINTER(c_size_t), POINTER(c_size_t)]),
    "kvq_append": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32, c_int32,
                             c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "kvq_decode_num_splits": (c_int32, [POINTER(kvq_cache_desc), c_int32, c_int32, c_int32,
                                        c_int32]),
    "kvq_decode_workspace_size": (c_size_t, [POINTER(kvq_cache_desc), c_int32, c_int32,
                                             c_int32, c_int32]),
    "kvq_decode_attn": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32, c_int32,
                                  c_void_p, c_void_p, c_int32, c_int32, c_float, c_void_p,
                                  c_void_p, c_size_t, c_void_p, c_void_p]),
    "kvq_append_decode_attn": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32,
                                         c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32,
                                         c_int32, c_float, c_void_p, c_void_p, c_size_t, c_void_p,
                                         c_void_p]),
    "kvq_decode_attn_static_ws": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32,
                                            c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                            c_float, c_void_p, c_void_p, c_void_p]),
    "kvq_rope_init": (c_int32, [POINTER(kvq_rope_desc), POINTER(kvq_rope)]),
    "kvq_rope_apply": (c_int32, [POINTER(kvq_rope), c_int32, c_int32, c_int32, c_int32, c_void_p,
                                 c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p]),
    "kvq_rope_append": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), POINTER(kvq_rope),
                                  c_int32, c_int32, c_void_p, c_void_p, c_int32, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "kvq_rope_axes_init": (c_int32, [POINTER(kvq_rope_axes_desc), POINTER(kvq_rope_axes)]),
    "kvq_rope_axes_apply": (c_int32, [POINTER(kvq_rope_axes), c_int32, c_int32, c_int32, c_int32,
                                      c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p]),
    "kvq_rope_axes_append": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache),
                                       POINTER(kvq_rope_axes), c_int32, c_int32, c_void_p,
                                       c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p]),
    "kvq_cache_read": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32, c_int32,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "kvq_extend_num_splits": (c_int32, [POINTER(kvq_cache_desc), c_int32, c_int32, c_int32,
                                        c_int32, c_int32]),
    "kvq_extend_workspace_size": (c_size_t, [POINTER(kvq_cache_desc), c_int32, c_int32, c_int32,
                                             c_int32, c_int32]),
    "kvq_extend_attn": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32, c_int32,
                                  c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                  c_float, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "kvq_pages_workspace_size": (c_size_t, [POINTER(kvq_page_pool)]),
    "kvq_pages_reorder": (c_int32, [POINTER(kvq_page_pool), c_void_p, c_void_p, c_void_p,
                                    c_void_p]),
    "kvq_pages_reserve": (c_int32, [POINTER(kvq_page_pool), c_void_p, c_void_p, c_int32, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "kvq_pages_compact": (c_int32, [POINTER(kvq_page_pool), c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_size_t, c_void_p, c_void_p]),
    "kvq_pages_copy": (c_int32, [POINTER(kvq_cache_desc), c_void_p, c_int32, c_void_p,
                                 c_void_p, c_int32, c_void_p, c_void_p]),
    "kvq_prefix_plan_size": (c_size_t, [c_int32, c_int32]),
    "kvq_prefix_plan": (c_int32, [c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_size_t,
                                  c_void_p, c_void_p]),
    "kvq_prefix_find_workspace_size": (c_size_t, [POINTER(kvq_page_pool)]),
    "kvq_prefix_find": (c_int32, [POINTER(kvq_page_pool), c_void_p, c_int32, c_int32, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_size_t, c_void_p, c_void_p]),
    "kvq_prefix_attn_workspace_size": (c_size_t, [POINTER(kvq_cache_desc), POINTER(kvq_cache_desc),
                                                  c_int32, c_int32, c_int32, c_int32, c_int32,
                                                  c_int32, c_int32, c_int32]),
    "kvq_prefix_attn": (c_int32, [POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32,
                                  POINTER(kvq_cache_desc), POINTER(kvq_cache), c_int32, c_int32,
                                  c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                  c_int32, c_int32, c_int32, c_int32, c_float, c_void_p, c_void_p,
                                  c_size_t, c_void_p, c_void_p]),
    "kvq_debug_checks": (c_int32, []),
    "kvq_debug_shrink_extent": (c_int32, [c_int32, c_int64]),
    "kvq_debug_fail_wait": (c_int32, [c_int32, c_int32]),
    "kvq_status_string": (ctypes.c_char_p, [c_int32]),
}


def load(path: str) -> ctypes.CDLL:
    """A handle on the library at `path` with the C signatures attached."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{os.path.basename(path)} is not built; run `python -m quantized_kv_decode_gb300.build` "
            "(the library has no fallback path)")
    handle = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


def lib() -> ctypes.CDLL:
    """Load libkvq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def use(handle: ctypes.CDLL | None) -> ctypes.CDLL | None:
    """Route the binding's calls to `handle` (e.g. the debug build,
    libkvq_debug.so); None returns to libkvq.so.  Returns the previous handle."""
    global _lib
    prev, _lib = _lib, handle
    return prev


def status_string(status: int) -> str:
    return lib().kvq_status_string(int(status)).decode()


def check(status: int, where: str) -> None:
    if status != KVQ_OK:
        raise KVQError(status, where)
