"""ctypes loader for libvta_gb300.so (the C ABI of include/rpe_attn.h).

Loading fails loudly when the library has not been built: there is no CPU
or pure-PyTorch stand-in for any entry point.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libvta_gb300.so")
BIND_PATH = os.path.join(_PKG, "_build", "vta_bind.so")

RPE_OK = 0
RPE_ERR_INVALID_ARG = 1
RPE_ERR_UNSUPPORTED = 2
RPE_ERR_CUDA = 3
RPE_ERR_TIMEOUT = 4
RPE_MAP_PRODUCT = 0
RPE_MAP_EUCLIDEAN = 1
RPE_MAP_CROSS = 2
RPE_MAP_CLIP_PRODUCT = 3
RPE_TERM_K, RPE_TERM_Q, RPE_TERM_V = 1, 2, 4
RPE_TABLES_CROSS = 8
RPE_TABLES_PER_HEAD = 16
RPE_CLS_TOKEN = 32
RPE_DTYPE_BF16, RPE_DTYPE_F32, RPE_DTYPE_F16 = 0, 1, 2
RPE_ROPE_NONE, RPE_ROPE_LINEAR, RPE_ROPE_NTK, RPE_ROPE_BANDS, RPE_ROPE_YARN = 0, 1, 2, 3, 4
RPE_ROPE_INTERLEAVED, RPE_ROPE_INVERSE, RPE_ROPE_BATCH_POSITIONS = 1, 2, 4
RPE_NORM_RMS, RPE_NORM_LAYER = 0, 1
RPE_ATTN_CAUSAL = 1


class View(ctypes.Structure):
    """rpe_view: a [batch, tokens, heads, d] tensor with element strides."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


# name -> (restype, argtypes) for every symbol the header declares
_f, _i64, _view = ctypes.c_float, ctypes.c_int64, ctypes.POINTER(View)
_i, _u, _d, _p, _u64 = ctypes.c_int, ctypes.c_uint, ctypes.c_double, ctypes.c_void_p, ctypes.c_uint64
SIGNATURES = {
    "rpe_build_bucket_ids": (_i, [_i, _i, _i, _d, _d, _d, _p, _p, ctypes.POINTER(_i), _p]),
    "rpe_attn_fwd": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _u, _i, _p, _p]),
    "swin_window_attn_fwd": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p]),
    "swin_window_attn_fwd_noalloc": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _p]),
    "swin_noalloc_status": (_i, [ctypes.POINTER(_u), _i]),
    "swin_noalloc_status_word": (_i, [ctypes.POINTER(_p)]),
    "swin_window_attn_fwd_fmap": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p]),
    "rpe_attn_bias_fwd": (_i, [_p, _p, _p, _p, _i, _p, _i, ctypes.c_uint, _i, _i, _i, _i, _i, _i,
                               _p, _p]),
    "rope_build_phases": (_i, [_i, _i, _i, _d, _d, _d, _d, _d, _p, ctypes.POINTER(_f), _p]),
    "rope_fwd": (_i, [_view, _view, _view, _view, _p, _i, _p, _i, _f, _u, _i64, _i64, _i, _i, _i,
                      _i, _p]),
    "qk_norm_rope_fwd": (_i, [_view, _view, _view, _view, _i, _f, _p, _p, _i, _p, _i, _p, _i, _f,
                              _u, _i64, _i64, _i, _i, _i, _i, _p]),
    "packed_attn_fwd": (_i, [_view, _view, _view, _view, _p, _p, _p, _p, _i, _i64, _i64, _i, _i,
                             _i, _f, _u, _i, _p, ctypes.c_size_t, _p]),
    "packed_attn_workspace": (_i, [_i64, _i64, _i, _i, _i, _i, _i,
                                   ctypes.POINTER(ctypes.c_size_t)]),
    "rpe_device_status": (_i, [ctypes.POINTER(_u), _i]),
    "rpe_wait_probe": (_i, [_u64, _p]),
    "rpe_status_string": (ctypes.c_char_p, [_i]),
    "rpe_release_stream": (_i, [_p]),
    "rpe_shutdown": (_i, []),
}

_lib = None


class RpeError(RuntimeError):
    def __init__(self, fn, status):
        msg = lib().rpe_status_string(status).decode()
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


def lib():
    """The loaded library; raises if it was never built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m vision_transformer_attention_gb300.build` (no CPU fallback exists)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


class _NoBind:
    """Stands for vta_bind where it cannot be loaded: nothing is done the quick way."""
    rope = attn = staticmethod(lambda *args: None)


_bind = None


def bind():
    """The extension module that makes the calls on tokens straight from tensor objects
    (csrc/bind.cpp); its functions return None for a call that they leave to api.py."""
    global _bind
    if _bind is None:
        lib()
        try:
            import torch  # noqa: F401  (its libraries are what the module links against)
            spec = importlib.util.spec_from_file_location("vta_bind", BIND_PATH)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _bind = module
        except (ImportError, OSError, AttributeError):
            _bind = _NoBind
    return _bind


def check(fn, status):
    if status != RPE_OK:
        raise RpeError(fn, status)
