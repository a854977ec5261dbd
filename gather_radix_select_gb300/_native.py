"""ctypes binding of libsel.so (include/sel.h, include/sel/*.h).  Argument marshalling only.  (The calls of
include/sel/cache_serving.h go by a compiled module, ``binding()``: csrc/binding.cpp says why.)

The library is built in-tree by ``gather_radix_select_gb300.build``; loading
fails loudly (``RuntimeError``) when it is missing -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from . import build as _build

SEL_OK, SEL_EINVAL, SEL_EALIGN, SEL_EUNSUPPORTED, SEL_ECUDA, SEL_ETIMEOUT, SEL_ESCRATCH, SEL_EBOUNDS = range(8)
SEL_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024
SEL_F32, SEL_BF16 = 0, 1
SEL_E4M3 = 2                 # include/sel/cache.h
SEL_CACHE_GROUP = 128
SEL_CACHE_ATTN_MAX_D = 512
SEL_I32, SEL_I64 = 0, 1
SEL_MAX_K = 4096
# include/sel_tuning.h
SEL_TUNE_PLAN, SEL_TUNE_PARTS, SEL_TUNE_ROW_SAMPLE, SEL_TUNE_HIST_AGG, SEL_TUNE_ROW_ORDER = range(5)
SEL_PLANS = {"auto": -1, "reg": 0, "row": 1, "wide": 2, "split": 3, "stream": 4, "flat": 5}

# every symbol the headers under include/ declare, with its ctypes signature
_vp, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class SelCache(ctypes.Structure):
    """sel_cache of include/sel/cache.h."""
    _fields_ = [("data", _vp), ("scales", _vp), ("dtype", _int), ("pages", _i64), ("page_size", _i64), ("d", _i64),
                ("page_stride", _i64), ("row_stride", _i64), ("scale_page_stride", _i64),
                ("scale_row_stride", _i64)]


class SelRotation(ctypes.Structure):
    """sel_rotation of include/sel/cache_serving.h."""
    _fields_ = [("table", _vp), ("positions", _i64), ("stride", _i64), ("first", _i64), ("rot", _i64),
                ("interleaved", _int)]


_cache_p, _rotation_p = ctypes.POINTER(SelCache), ctypes.POINTER(SelRotation)
SIGNATURES = {
    "sel_stride_requirement": (_int, [ctypes.POINTER(_int), ctypes.POINTER(_int)]),
    "sel_topk": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _int, _int, _int, _int,
                        _vp, _i64, _vp, _i64, _vp, ctypes.c_size_t, _vp, _vp, _vp]),
    "sel_topk_workspace_size": (ctypes.c_size_t, [_int, _i64, _i64, _int]),
    "sel_max_cols": (_i64, [_int]),
    "sel_gather_rows": (_int, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _int, _i64, _i64, _i64,
                               _vp, _vp, _vp]),
    "sel_gather_rows_pair": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _int,
                                    _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "sel_block_topk_gather": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _int, _i64, _vp, _i64,
                                     _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                     _vp, ctypes.c_size_t, _vp, _vp, _vp]),
    "sel_topk_gather": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _int, _int, _int, _int,
                               _vp, _i64, _vp, _i64,
                               _vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp,
                               _vp, ctypes.c_size_t, _vp, _vp, _vp]),
    "sel_topk_noalloc": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _int, _int, _int, _int,
                                _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "sel_strerror": (ctypes.c_char_p, [_int]),
    "sel_topk_kernel_name": (ctypes.c_char_p, [_int, _i64, _i64, _int, _i64]),
    "sel_set_tuning": (_int, [_int, _int]),
    "sel_get_tuning": (_int, [_int]),
    "sel_selftest_wait_timeout": (_int, [_vp, ctypes.c_longlong, _vp]),
    "sel_debug_build": (_int, []),
    "sel_cache_write": (_int, [_vp, _int, _i64, _i64, _vp, _int, _cache_p, _vp, _vp]),
    "sel_cache_gather": (_int, [_cache_p, _vp, _i64, _i64, _i64, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "sel_cache_attention": (_int, [_vp, _i64, _i64, _i64, _i64, _cache_p, _vp, _i64, _i64, _i64, _vp, _vp, _int,
                                   _i64, _i64, _i64, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]),
    "sel_cache_set_wait_limit": (_int, [_i64]),
    "sel_cache_append": (_int, [_vp, _int, _i64, _i64, _cache_p, _vp, _i64, _i64, _i64, _vp, _int, _rotation_p, _vp,
                                _int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "sel_cache_attention_window": (_int, [_vp, _i64, _i64, _i64, _i64, _cache_p, _vp, _i64, _i64, _i64, _vp, _i64,
                                          _i64, _i64, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]),
    "sel_cache_attention_window_workspace_size": (ctypes.c_size_t, [_i64] * 9),
    "sel_cache_attention_shared": (_int, [_vp, _i64, _i64, _i64, _i64, _cache_p, _vp, _i64, _i64, _i64, _vp, _i64,
                                          _i64, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]),
    "sel_cache_attention_shared_workspace_size": (ctypes.c_size_t, [_i64] * 8),
    "sel_cache_attention_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64, _i64, _i64, _i64, _i64, _int, _i64]),
}

_lock = threading.Lock()
_lib = None


def library_path() -> str:
    """libsel.so, or the bounds-checked libsel_debug.so when SEL_LIBRARY=debug is set (read when the
    library is first loaded)."""
    return _build.DEBUG_SO if os.environ.get("SEL_LIBRARY", "") == "debug" else _build.SO


def load(build_if_missing: bool = False):
    """Load libsel.so once.  Raises RuntimeError when it is not built."""
    global _lib
    if _lib is not None:  # (without the lock: set once, when the library is complete)
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(
                    "libsel.so is not built (%s); run `python -m gather_radix_select_gb300.build`" % path)
            _build.build(debug=path == _build.DEBUG_SO)
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


_binding = None


def binding():
    """The module of csrc/binding.cpp, bound to the loaded library.  Raises RuntimeError when it is not built."""
    global _binding
    if _binding is not None:
        return _binding
    lib = load()
    with _lock:
        if _binding is None:
            path = _build.binding_path()
            if not os.path.exists(path):
                raise RuntimeError("%s is not built; run `python -m gather_radix_select_gb300.build`" % path)
            loader = importlib.machinery.ExtensionFileLoader("_binding", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
            module.bind(lib._handle)
            _binding = module
        return _binding


class SelError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = load().sel_strerror(status).decode()
        super().__init__("%s failed: %s (status %d)" % (where, msg, status))
        self.status = status


def check(status: int, where: str) -> None:
    if status != SEL_OK:
        raise SelError(status, where)
