"""Python binding of libnvfp4moe.so, the NVFP4 weight-only MoE library for
B200 (sm_100a), and of libnvfp4dense.so, the dense feed-forward operators next
to it.

Two layers:
  * the C ABI under its own names (`nvfp4_quantize`, `moe_route`,
    `moe_nvfp4_forward`, ... in `nvfp4_weight_only_router_b200.capi`): raw
    device pointers and sizes, returning the status code;
  * torch conveniences (`quantize`, `dequantize`, `route`, `permute`,
    `MoeLayer`, `residual_rmsnorm`): they allocate outputs and workspaces with torch and
    pass pointers to the same C calls on torch's current stream;
  * the dense operators in the same two layers (`dense_capi`; `mxfp4_quantize`,
    `mxfp4_linear`, `mxfp4_linear_a4`, `gated_ffn`, ...).

Every computation runs in the library's CUDA kernels; there is no fallback.
The shared library is loaded on first use of anything but `build`; that use
raises ImportError if it has not been built
(`python -m nvfp4_weight_only_router_b200.build`).
"""
from __future__ import annotations

import importlib

_API = {"MoeLayer", "MoeBlock", "DenseParts", "Aff4Experts", "Aff4Layer", "W4A4Layer", "Router", "Experts", "quantize", "dequantize", "route", "permute", "residual_rmsnorm",
        "device_status", "forward_views", "unscaled_hidden"}
_DENSE = {"Mxfp4Weight", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear", "mxfp4_linear_a4", "gated_ffn",
          "gated_ffn_forward", "gated_ffn_backward"}
_CAPI = {"NVFP4Error", "check", "status_string"}

__all__ = sorted(_API | _DENSE | _CAPI | {"capi", "dense_capi", "build"})


def __getattr__(name):
    if name in ("capi", "dense_capi"):
        return importlib.import_module("." + name, __name__)
    for names, module in ((_DENSE, ".dense"), (_CAPI, ".capi"), (_API, ".api")):
        if name in names:
            value = getattr(importlib.import_module(module, __name__), name)
            globals()[name] = value  # found at once from now on
            return value
    raise AttributeError(name)
