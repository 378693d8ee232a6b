"""The dense feed-forward library without a GPU: exported symbols, refusals
before anything is enqueued, and the 64-bit forms that the GPU tests compare
with (against each other and against differences)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from tests import dense_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096


@pytest.fixture(scope="module")
def dc():
    from nvfp4_weight_only_router_b200 import build
    build.build()
    from nvfp4_weight_only_router_b200 import dense_capi
    return dense_capi


@pytest.fixture(scope="module")
def codes(dc):
    from nvfp4_weight_only_router_b200 import capi
    return capi


def test_exports_are_the_header(dc):
    src = open(os.path.join(ROOT, "include", "nvfp4dense.h")).read()
    names = set(re.findall(r"NVFP4DENSE_API\s+[\w\s\*]+?\b(\w+)\s*\(", src))
    out = os.popen(f"nm -D --defined-only {dc.LIB_PATH}").read().split("\n")
    assert names == {ln.split()[-1] for ln in out if " T " in ln} == set(dc.SIGNATURES)
    assert dc.nvfp4dense_abi_version() == 1
    assert dc.lib.nvfp4dense_last_cuda_error().decode() == "no error"


def test_quantize_refusals(dc, codes):
    q = dc.mxfp4_quantize
    assert q(P, 0, -1, 32, 32, P, P, None) == codes.NVFP4_ERR_INVALID_ARG
    assert q(P, 0, 1, 0, 32, P, P, None) == codes.NVFP4_ERR_INVALID_ARG
    assert q(P, 3, 1, 32, 32, P, P, None) == codes.NVFP4_ERR_INVALID_ARG
    assert q(None, 0, 1, 32, 32, P, P, None) == codes.NVFP4_ERR_INVALID_ARG
    assert q(P, 0, 2, 32, 31, P, P, None) == codes.NVFP4_ERR_INVALID_ARG
    assert q(P, 0, 1, 1 << 24, 1 << 24, P, P, None) == codes.NVFP4_ERR_UNSUPPORTED
    assert q(P, 0, 1 << 31, 32, 32, P, P, None) == codes.NVFP4_ERR_UNSUPPORTED
    assert q(P + 1, 0, 1, 32, 32, P, P, None) == codes.NVFP4_ERR_ALIGNMENT
    assert q(P + 2, 2, 1, 32, 32, P, P, None) == codes.NVFP4_ERR_ALIGNMENT
    assert q(P, 0, 1, 32, 32, P + 8, P, None) == codes.NVFP4_ERR_ALIGNMENT
    assert q(None, 0, 0, 32, 32, None, None, None) == codes.NVFP4_OK
    d = dc.mxfp4_dequantize
    assert d(P, P, 1, 32, P, 1, None) == codes.NVFP4_ERR_UNSUPPORTED
    assert d(P, P, 1, 32, None, 2, None) == codes.NVFP4_ERR_INVALID_ARG
    assert d(P, P, 1, 32, P + 4, 2, None) == codes.NVFP4_ERR_ALIGNMENT
    assert d(P, P, 1, 32, P, 7, None) == codes.NVFP4_ERR_INVALID_ARG
    assert d(None, None, 0, 32, None, 2, None) == codes.NVFP4_OK


def _w(dc, N=64, K=64, c=P, s=P):
    return dc.mxfp4_weight(c, s, N, K)


@pytest.mark.parametrize("a4", [False, True])
def test_linear_refusals(dc, codes, a4):
    call = dc.mxfp4_linear_a4 if a4 else dc.mxfp4_linear
    size = dc.mxfp4_linear_a4_workspace_bytes if a4 else dc.mxfp4_linear_workspace_bytes
    c = codes
    w = _w(dc)
    big = 1 << 30

    def run(x=P, dtype=0, ldx=64, T=4, w=w, act=0, y=P, ws=P, n=big):
        return call(x, dtype, ldx, T, ctypes.byref(w), act, y, ws, n, None)

    assert call(P, 0, 64, 4, None, 0, P, P, big, None) == c.NVFP4_ERR_INVALID_ARG
    assert run(T=-1) == run(x=None) == run(y=None) == run(dtype=5) == run(act=3) == c.NVFP4_ERR_INVALID_ARG
    assert run(ldx=56) == run(w=_w(dc, c=None)) == run(w=_w(dc, N=0)) == c.NVFP4_ERR_INVALID_ARG
    assert run(dtype=2) == c.NVFP4_ERR_UNSUPPORTED
    if not a4:
        assert run(dtype=1) == c.NVFP4_ERR_UNSUPPORTED
    for bad in (_w(dc, N=60), _w(dc, K=48), _w(dc, N=1 << 19), _w(dc, K=1 << 19)):
        assert run(w=bad) == c.NVFP4_ERR_UNSUPPORTED
        assert size(4, ctypes.byref(bad), 0) == 0
    assert run(w=_w(dc, N=72), act=1) == c.NVFP4_ERR_UNSUPPORTED      # halves of 36 rows
    assert run(T=(1 << 20) + 1) == c.NVFP4_ERR_UNSUPPORTED
    assert run(x=P + 2) == run(y=P + 8) == run(ldx=68) == run(w=_w(dc, s=P + 4)) == c.NVFP4_ERR_ALIGNMENT
    assert run(ws=P + 16) == c.NVFP4_ERR_ALIGNMENT
    assert size(4, ctypes.byref(w), 0) == 256                           # few tokens: none is used
    n = size(5000, ctypes.byref(w), 0)
    assert n > 256
    assert run(T=5000, n=n - 1) == run(T=5000, ws=None) == c.NVFP4_ERR_WORKSPACE
    assert run(T=0, x=None, y=None) == c.NVFP4_OK


def _f(dc, H=64, I=64, act=1, dtype=0, p=P):
    return dc.gated_ffn_weights(p, P, P, H, I, act, dtype)


def test_ffn_refusals(dc, codes):
    c = codes
    big = 1 << 30

    def fwd(x=P, ldx=64, T=4, f=None, y=P, saved=None, ws=P, n=big):
        return dc.gated_ffn_forward(x, ldx, T, ctypes.byref(f or _f(dc)), y, saved, ws, n, None)

    def bwd(dy=P, lddy=64, x=P, ldx=64, saved=P, T=4, f=None, outs=(P, P, P, P), ws=P, n=big):
        return dc.gated_ffn_backward(dy, lddy, x, ldx, saved, T, ctypes.byref(f or _f(dc)), *outs, ws, n, None)

    for run in (fwd, bwd):
        assert run(T=-1) == run(x=None) == run(ldx=56) == c.NVFP4_ERR_INVALID_ARG
        assert run(f=_f(dc, p=None)) == run(f=_f(dc, H=0)) == run(f=_f(dc, act=4)) == c.NVFP4_ERR_INVALID_ARG
        assert run(f=_f(dc, act=0)) == run(f=_f(dc, dtype=2)) == c.NVFP4_ERR_UNSUPPORTED
        assert run(f=_f(dc, H=60)) == run(f=_f(dc, I=68)) == run(T=(1 << 20) + 1) == c.NVFP4_ERR_UNSUPPORTED
        assert run(x=P + 8) == run(ldx=68) == run(f=_f(dc, p=P + 2)) == run(ws=P + 16) == c.NVFP4_ERR_ALIGNMENT
        assert run(ws=None) == run(n=0) == c.NVFP4_ERR_WORKSPACE
    assert fwd(saved=P + 8) == fwd(y=P + 2) == c.NVFP4_ERR_ALIGNMENT
    assert bwd(dy=None) == bwd(saved=None) == bwd(lddy=32) == c.NVFP4_ERR_INVALID_ARG
    assert bwd(outs=(P, P, P + 8, P)) == bwd(lddy=68) == c.NVFP4_ERR_ALIGNMENT
    assert fwd(T=0, x=None, y=None) == c.NVFP4_OK
    assert bwd(outs=(None,) * 4, T=0) == c.NVFP4_OK
    n = dc.gated_ffn_backward_workspace_bytes(100, ctypes.byref(_f(dc)))
    assert bwd(T=100, n=n - 1) == c.NVFP4_ERR_WORKSPACE
    assert bwd(saved=P + 16) == c.NVFP4_ERR_ALIGNMENT
    # h in 16 bits with rows of whole 128-byte lines, and blocks of 32 rows x 16 hidden units in 2 x 24
    assert dc.gated_ffn_saved_bytes(100, ctypes.byref(_f(dc))) == 12800 + 4 * 4 * (32 * 16 * 6)
    assert dc.gated_ffn_saved_bytes(3, ctypes.byref(_f(dc, I=8))) == 512 + 32 * 16 * 6
    assert dc.gated_ffn_saved_bytes(0, ctypes.byref(_f(dc))) == 256
    assert dc.gated_ffn_saved_bytes(100, ctypes.byref(_f(dc, I=4))) == 0
    assert dc.gated_ffn_backward_workspace_bytes(100, ctypes.byref(_f(dc, I=4))) == 0


def test_python_refusals(dc):
    import nvfp4_weight_only_router_b200 as lib
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    for call in (lambda: lib.mxfp4_quantize(x), lambda: lib.mxfp4_quantize(x.int()),
                 lambda: lib.Mxfp4Weight(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), 64),
                 lambda: lib.gated_ffn_forward(x, w, w, w.T.contiguous()),
                 lambda: lib.gated_ffn_forward(x, w, w, w), lambda: lib.gated_ffn(x, w, w, w.T, "relu")):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------ the 64-bit forms
def test_encodings_agree():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 100)) * np.exp2(rng.integers(-40, 40, (6, 1)))
    x[0, :32] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6.5, 7.99, -5, -2.5, 0, -0.0, 4, 6, 1] * 2)
    x[1, 32:64] = 0
    q, s = R.mx_encode(x)
    v = R.mx_decode(q, s, 100)
    assert np.array_equal(v, R.mx_round(torch.from_numpy(x)).numpy())
    # a second rounding keeps the values
    assert np.array_equal(R.mx_decode(*R.mx_encode(v), 100), v)
    # ties to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert v[0, :9].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6]


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_gradients_against_differences(act):
    gen = torch.Generator().manual_seed(1)
    T, H, I = 5, 8, 6
    t = [torch.randn(s, generator=gen, dtype=torch.float64) for s in ((T, H), (I, H), (I, H), (H, I), (T, H))]
    x, gate, up, down, dy = t
    out = R.ffn64(x, gate, up, down, dy, act, torch.bfloat16)
    eps = 1e-5
    for name, k in (("dx", 0), ("dgate", 1), ("dup", 2), ("ddown", 3)):
        d = torch.randn(t[k].shape, generator=gen, dtype=torch.float64)
        ends = []
        for s in (eps, -eps):
            moved = list(t[:4])
            moved[k] = moved[k] + s * d
            ends.append((R.ffn64(*moved, None, act, torch.bfloat16)["y"][0] * dy).sum())
        # central differences: relative error of order eps^2 plus rounding 1e-16 / eps
        diff, form = (ends[0] - ends[1]) / (2 * eps), (out[name][0] * d).sum()
        assert abs(diff - form) <= 1e-7 * max(1.0, abs(form)), (name, diff, form)
