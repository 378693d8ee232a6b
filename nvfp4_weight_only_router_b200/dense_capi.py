"""ctypes declarations of the C ABI in include/nvfp4dense.h (argument
marshalling only), in the manner of `capi`: C names and signatures, pointers
as Python ints, each call returning the nvfp4_status code."""
from __future__ import annotations

import ctypes
import os

from . import capi
from .capi import NVFP4_OK, NVFP4Error, c_int32, c_int64, c_size_t, c_void_p

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4dense.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m nvfp4_weight_only_router_b200.build` "
        "(the package has no fallback path)")
lib = ctypes.CDLL(LIB_PATH)

BF16, F16, F32 = 0, 1, 2
ACT_NONE, ACT_GELU_TANH, ACT_SILU = 0, 1, 2


class mxfp4_weight(ctypes.Structure):
    _fields_ = [("codes", c_void_p), ("scales", c_void_p), ("N", c_int32), ("K", c_int32)]


class gated_ffn_weights(ctypes.Structure):
    _fields_ = [("gate", c_void_p), ("up", c_void_p), ("down", c_void_p), ("H", c_int32), ("I", c_int32),
                ("act", c_int32), ("dtype", c_int32)]


_W = ctypes.POINTER(mxfp4_weight)
_F = ctypes.POINTER(gated_ffn_weights)
_LINEAR = [c_void_p, c_int32, c_int64, c_int32, _W, c_int32, c_void_p, c_void_p, c_size_t, c_void_p]

# name -> (restype, argtypes), in the order of the header
SIGNATURES = {
    "mxfp4_quantize": (c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p]),
    "mxfp4_dequantize": (c_int32, [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_int32, c_void_p]),
    "mxfp4_linear_workspace_bytes": (c_size_t, [c_int32, _W, c_int32]),
    "mxfp4_linear": (c_int32, _LINEAR),
    "mxfp4_linear_a4_workspace_bytes": (c_size_t, [c_int32, _W, c_int32]),
    "mxfp4_linear_a4": (c_int32, _LINEAR),
    "gated_ffn_saved_bytes": (c_size_t, [c_int32, _F]),
    "gated_ffn_forward_workspace_bytes": (c_size_t, [c_int32, _F]),
    "gated_ffn_forward": (c_int32, [c_void_p, c_int64, c_int32, _F, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "gated_ffn_backward_workspace_bytes": (c_size_t, [c_int32, _F]),
    "gated_ffn_backward": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32, _F, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "nvfp4dense_get_device_status": (c_int32, [c_void_p]),
    "nvfp4dense_last_cuda_error": (ctypes.c_char_p, []),
    "nvfp4dense_abi_version": (ctypes.c_int, []),
}

for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args
    globals()[_name] = _fn


def check(status: int, what: str) -> None:
    if status != NVFP4_OK:
        text = lib.nvfp4dense_last_cuda_error().decode() if status == capi.NVFP4_ERR_CUDA else None
        raise NVFP4Error(status, what, text)
