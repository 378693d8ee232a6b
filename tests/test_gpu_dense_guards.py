"""Out-of-bounds writes of the dense library: every output, kept block and workspace
of a call sits between guard regions, which the call must leave unchanged; and what
such a buffer held before the call changes no result."""
import ctypes

import pytest
import torch

import nvfp4_weight_only_router_b200 as lib
from nvfp4_weight_only_router_b200 import dense_capi as dc
from tests.test_gpu_guards import Guarded, _stream

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPE = {BF: dc.BF16, F16: dc.F16, F32: dc.F32}


def _twice(dev, sizes, call):
    """call(pointers) with buffers that held 0xA5 and 0xFF before; the contents agree."""
    results = []
    for fill in (0xA5, 0xFF):
        bufs = {k: Guarded(n, dev) for k, n in sizes.items()}
        for b in bufs.values():
            b.buf[4096:4096 + b.n] = fill
        dc.check(call({k: b.ptr for k, b in bufs.items()}), "call")
        assert lib.device_status() == 0
        for k, b in bufs.items():
            b.check(k)
        results.append({k: b.buf[4096:4096 + b.n].clone() for k, b in bufs.items()})
    return results


def _same(results, *names):
    for k in names:
        assert torch.equal(results[0][k], results[1][k]), k


def _randn(dev, dtype, *shape, k=1.0, seed=0):
    return (torch.randn(shape, generator=torch.Generator(dev).manual_seed(seed), device=dev) * k).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 33), (7, 257), (129, 2101), (3000, 100), (2500, 2112)])
def test_quantize_and_back(dev, dtype, rows, K):
    x = _randn(dev, dtype, rows, K)
    nb = -(-K // 32)
    r = _twice(dev, {"codes": rows * 16 * nb, "scales": rows * nb}, lambda p: dc.mxfp4_quantize(
        x.data_ptr(), TYPE[dtype], rows, K, K, p["codes"], p["scales"], _stream()))
    _same(r, "codes", "scales")
    codes, scales = r[0]["codes"], r[0]["scales"]
    for t in (F32, BF):
        r = _twice(dev, {"out": rows * K * t.itemsize}, lambda p: dc.mxfp4_dequantize(
            codes.data_ptr(), scales.data_ptr(), rows, K, p["out"], TYPE[t], _stream()))
        _same(r, "out")


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("N,K", [(16, 32), (208, 160), (2816, 704)])
@pytest.mark.parametrize("T", [1, 9, 33, 129, 300, 520])
def test_linear(dev, T, N, K, act):
    weight = lib.Mxfp4Weight.quantize(_randn(dev, BF, N, K, k=K ** -0.5))
    w = dc.mxfp4_weight(weight.codes.data_ptr(), weight.scales.data_ptr(), N, K)
    for call, size, types in ((dc.mxfp4_linear, dc.mxfp4_linear_workspace_bytes, (BF,)),
                              (dc.mxfp4_linear_a4, dc.mxfp4_linear_a4_workspace_bytes, (BF, F16))):
        n = size(T, ctypes.byref(w), act)
        for t in types:
            x = _randn(dev, t, T, K, seed=T)
            r = _twice(dev, {"y": T * (N // 2 if act else N) * 2, "ws": n}, lambda p: call(
                x.data_ptr(), TYPE[t], K, T, ctypes.byref(w), act, p["y"], p["ws"], n, _stream()))
            _same(r, "y")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (3, 136, 72), (16, 264, 512), (33, 72, 200), (130, 520, 264), (257, 200, 1000)])
def test_gated_ffn(dev, T, H, I, dtype):
    x, dy = _randn(dev, dtype, T, H), _randn(dev, dtype, T, H, seed=1)
    gate, up, down = (_randn(dev, dtype, *s, k=s[1] ** -0.5, seed=2 + i) for i, s in enumerate(((I, H), (I, H), (H, I))))
    f = dc.gated_ffn_weights(gate.data_ptr(), up.data_ptr(), down.data_ptr(), H, I, dc.ACT_SILU, TYPE[dtype])
    ref = ctypes.byref(f)
    n = dc.gated_ffn_forward_workspace_bytes(T, ref)
    _same(_twice(dev, {"y": T * H * 2, "ws": n}, lambda p: dc.gated_ffn_forward(
        x.data_ptr(), H, T, ref, p["y"], None, p["ws"], n, _stream())), "y")
    kept = dc.gated_ffn_saved_bytes(T, ref)
    r = _twice(dev, {"y": T * H * 2, "saved": kept}, lambda p: dc.gated_ffn_forward(
        x.data_ptr(), H, T, ref, p["y"], p["saved"], None, 0, _stream()))
    _same(r, "y")
    # the padding of what is kept may hold anything: the gradients do not read it
    n = dc.gated_ffn_backward_workspace_bytes(T, ref)
    grads = []
    for one in r:
        saved = torch.empty(kept, dtype=torch.uint8, device=dev)
        saved.copy_(one["saved"])
        grads += _twice(dev, {"dx": T * H * 2, "dgate": I * H * 2, "dup": I * H * 2, "ddown": H * I * 2, "ws": n},
                        lambda p: dc.gated_ffn_backward(dy.data_ptr(), H, x.data_ptr(), H, saved.data_ptr(), T, ref,
                                                        p["dx"], p["dgate"], p["dup"], p["ddown"], p["ws"], n, _stream()))
    for other in grads[1:]:
        _same((grads[0], other), "dx", "dgate", "dup", "ddown")
