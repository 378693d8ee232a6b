"""Build the in-tree shared libraries libnvfp4moe.so (csrc/*.cu) and
libnvfp4dense.so (csrc/dense/*.cu and the host helpers it shares) for sm_100a
with nvcc, and _dense_calls.so (csrc/dense/torch_calls.cpp), torch's calls of
the latter, with g++.  The C libraries need no torch:
where it is not installed, torch's calls are left out.

    python -m nvfp4_weight_only_router_b200.build [--force] [--verbose]

Each source is compiled to an object under _build/ and linked into its
library in nvfp4_weight_only_router_b200/.  Sources are rebuilt when they or
any header is newer than their object.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnvfp4moe.so")
DENSE_LIB = os.path.join(PKG, "libnvfp4dense.so")
DENSE_CALLS = os.path.join(PKG, "_dense_calls.so")
DENSE_SHARED = ("host_util", "tma_map")  # csrc/*.cu that the dense library links too

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _headers() -> list[str]:
    return [h for d in (CSRC, os.path.join(CSRC, "dense")) for e in ("*.cuh", "*.h")
            for h in glob.glob(os.path.join(d, e))] + glob.glob(os.path.join(ROOT, "include", "*.h"))


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    flags = NVCC_FLAGS + (extra_flags or [])
    hdr_mtime = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    main = {src: _object(src) for src in sorted(glob.glob(os.path.join(CSRC, "*.cu")))}
    dense = {src: _object(src, "dense_") for src in sorted(glob.glob(os.path.join(CSRC, "dense", "*.cu")))}
    stale = [(src, obj) for src, obj in {**main, **dense}.items()
             if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_mtime)]
    calls = os.path.join(CSRC, "dense", "torch_calls.cpp")
    calls_obj = os.path.join(BUILD, "dense_torch_calls.o")
    abi = max(os.path.getmtime(f) for f in [calls] + glob.glob(os.path.join(ROOT, "include", "*.h")))
    with_torch = importlib.util.find_spec("torch") is not None
    with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        host = None
        if with_torch and (force or not os.path.exists(calls_obj) or os.path.getmtime(calls_obj) < abi):
            host = pool.submit(_compile_calls, calls, calls_obj, verbose)
        list(pool.map(lambda so: _compile(*so, flags, verbose), stale))
    _link(LIB, list(main.values()), force, verbose)
    _link(DENSE_LIB, list(dense.values()) + [_object(os.path.join(CSRC, n + ".cu")) for n in DENSE_SHARED], force, verbose)
    if not with_torch:
        print(f"torch is not installed: {os.path.basename(DENSE_CALLS)} is not built", file=sys.stderr)
        return LIB
    if host is not None:
        host.result()
    if force or not os.path.exists(DENSE_CALLS) or os.path.getmtime(calls_obj) > os.path.getmtime(DENSE_CALLS):
        _link_calls(calls_obj, verbose)
    return LIB


def _object(src: str, prefix: str = "") -> str:
    return os.path.join(BUILD, prefix + os.path.basename(src)[:-3] + ".o")


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def _compile(src: str, obj: str, flags: list[str], verbose: bool) -> None:
    _run([nvcc()] + (["-Xptxas=-v"] if verbose else []) + ARCH + flags + ["-c", src, "-o", obj], verbose)


def _link(lib: str, objs: list[str], force: bool, verbose: bool) -> None:
    if force or not os.path.exists(lib) or any(os.path.getmtime(o) > os.path.getmtime(lib) for o in objs):
        tmp = lib + ".tmp"
        _run([nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs, verbose)
        os.replace(tmp, lib)


def _compile_calls(src: str, obj: str, verbose: bool) -> None:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    inc = cpp_extension.include_paths("cuda") + [sysconfig.get_paths()["include"], _cuda_include()]
    _run(["g++", "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_dense_calls",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] +
         ["-isystem" + i for i in inc] + ["-c", src, "-o", obj], verbose)


def _cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")


def _link_calls(obj: str, verbose: bool) -> None:
    from torch.utils import cpp_extension
    tmp = DENSE_CALLS + ".tmp"
    libs = cpp_extension.library_paths()
    # libnvfp4dense.so is found next to the module
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:" + os.path.basename(DENSE_LIB), "-Wl,-rpath,$ORIGIN"] +
         ["-L" + p for p in libs] + ["-lc10", "-lc10_cuda", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"], verbose)
    os.replace(tmp, DENSE_CALLS)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
