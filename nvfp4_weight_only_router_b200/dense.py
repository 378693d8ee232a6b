"""torch conveniences over the dense feed-forward C ABI (include/nvfp4dense.h):
MXFP4 quantisation, products with MXFP4 weights, and the gated feed-forward
block with its backward pass.

Every function runs on torch's current stream of the tensors' device, or on
`stream`; outputs and workspaces are allocated on that stream, per call, so
that calls may overlap and be captured freely.  Tensors are [rows, features]
with contiguous features, on 16-byte boundaries (what is quantised: of its
elements); x (and dy) may be row-strided views.

A call on the current stream is made whole by `_dense_calls` (the same C calls,
with checks and allocations in C++: 5 us of host time instead of 9 to 18).  It
returns None where an argument does not fit or the call is refused, before
anything is enqueued; the steps that follow here then say what is wrong, and
serve calls on a given stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses

import torch
from torch.autograd import forward_ad

from . import capi
from . import dense_capi as dc
from .dense_capi import check

try:
    from . import _dense_calls as _calls  # after dense_capi, which loads its library
except ImportError as e:
    raise ImportError("_dense_calls is missing or was built for another torch: build it with "
                      "`python -m nvfp4_weight_only_router_b200.build --force`") from e

_DTYPE = {torch.bfloat16: dc.BF16, torch.float16: dc.F16, torch.float32: dc.F32}
_ACT = {None: dc.ACT_NONE, "gelu_tanh": dc.ACT_GELU_TANH, "silu": dc.ACT_SILU}
_VALUES = (torch.float32, torch.bfloat16)
_byref = ctypes.byref
_HERE = contextlib.nullcontext()


def _act(name, gated: bool = False) -> int:
    if name not in _ACT or (gated and name is None):
        raise ValueError(f"activation must be 'gelu_tanh' or 'silu'{'' if gated else ' or None'}, not {name!r}")
    return _ACT[name]


def _rows(t: torch.Tensor, what: str, features: int | None = None) -> int:
    """Checks a [rows, features] device tensor; its row stride in elements."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device")
    if t.dim() != 2 or (features is not None and t.shape[1] != features):
        raise ValueError(f"{what} must be a tensor [rows, {'features' if features is None else features}], "
                         f"not {list(t.shape)}")
    n, f = t.shape
    if f > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous features")
    if n <= 1:
        return f
    ld = t.stride(0)
    if ld < f:
        raise ValueError(f"{what} has overlapping rows")
    return ld


def _int32(name: str, *sizes: int) -> None:
    """Refuses sizes that the C call's 32-bit arguments cannot hold (ctypes would cut them)."""
    if max(sizes) > 0x7FFFFFFF:
        check(capi.NVFP4_ERR_UNSUPPORTED, name)


def _same(what: str, *tensors: torch.Tensor) -> None:
    a = tensors[0]
    for t in tensors[1:]:
        if t.dtype != a.dtype or t.device != a.device:
            raise ValueError(f"{what} must have one dtype and one device")


def _contiguous(what: str, *tensors: torch.Tensor) -> None:
    for t in tensors:
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")


def _on(stream, *tensors: torch.Tensor):
    """Context in which the call allocates and launches: the tensors' device,
    and `stream` if given (the tensors are then also held for it)."""
    if stream is not None:
        if stream.device != tensors[0].device:
            raise ValueError("stream and tensors are on different devices")
        for t in tensors:
            t.record_stream(stream)
        return torch.cuda.stream(stream)
    dev = tensors[0].get_device()
    return _HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev)


# the stream's handle, without a Stream object around it (1 us of a call's 10)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _bytes(n: int, t: torch.Tensor) -> torch.Tensor:
    """n (at least 256) bytes of workspace on t's device; 0 means arguments that the call refuses."""
    return t.new_empty(max(n, 256), dtype=torch.uint8)


class _Undifferentiated(torch.autograd.Function):
    """The output of `call`, computed from tensors that a graph is being recorded for:
    a backward pass that comes to it raises, instead of losing their gradients."""
    @staticmethod
    def forward(ctx, call, advice, *inputs):
        ctx.advice = advice
        return call()

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError(ctx.advice)


def _recorded(*tensors: torch.Tensor) -> bool:
    if forward_ad._current_level >= 0 and torch._C._is_fwd_grad_enabled():   # tensors may carry tangents
        return True
    for t in tensors:
        if t.requires_grad:
            return torch.is_grad_enabled()
    return False


# ------------------------------------------------------------------- MXFP4
def mxfp4_quantize(x: torch.Tensor, stream=None):
    """bf16, f16 or f32 [R, K] -> (codes uint8 [R, 16 ceil(K/32)], scales uint8
    [R, ceil(K/32)]): E2M1 codes under one power-of-two scale per 32 elements."""
    if stream is None:
        out = _calls.quantize(x)
        if out is not None:
            return out
    if x.dtype not in _DTYPE:
        raise ValueError("x must be bf16, f16 or f32")
    ld = _rows(x, "x")
    R, K = x.shape
    nb = (K + 31) // 32
    with _on(stream, x):
        codes, scales = x.new_empty((R, 16 * nb), dtype=torch.uint8), x.new_empty((R, nb), dtype=torch.uint8)
        check(dc.mxfp4_quantize(x.data_ptr(), _DTYPE[x.dtype], R, K, ld, codes.data_ptr(), scales.data_ptr(),
                                _raw_stream(x.get_device())), "mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, K: int | None = None, dtype=torch.float32,
                     stream=None) -> torch.Tensor:
    """The values [R, K] of codes and scales, in f32 or bf16 (K defaults to the
    whole blocks)."""
    if stream is None and dtype in _VALUES and (K is None or K > 0):
        out = _calls.dequantize(codes, scales, -1 if K is None else K, dtype is torch.bfloat16)
        if out is not None:
            return out
    _check_codes(codes, scales)
    R, nb = scales.shape
    K = 32 * nb if K is None else int(K)
    if (K + 31) // 32 != nb:
        raise ValueError(f"K = {K} does not have {nb} blocks of 32")
    if dtype not in _VALUES:
        raise ValueError("dtype must be float32 or bfloat16")
    with _on(stream, codes, scales):
        out = torch.empty((R, K), dtype=dtype, device=codes.device)
        check(dc.mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), R, K, out.data_ptr(), _DTYPE[dtype],
                                  _raw_stream(codes.get_device())), "mxfp4_dequantize")
    return out


def _check_codes(codes: torch.Tensor, scales: torch.Tensor) -> None:
    _rows(codes, "codes")
    _rows(scales, "scales")
    if codes.dtype != torch.uint8 or codes.shape != (scales.shape[0], 16 * scales.shape[1]):
        raise ValueError("codes must be uint8 [R, 16 B] for scales [R, B]")
    _same("codes and scales", codes, scales)
    _contiguous("codes and scales", codes, scales)


@dataclasses.dataclass(frozen=True, eq=False)
class Mxfp4Weight:
    """An MXFP4 weight matrix [N, K] on the device: codes uint8 [N, K/2] and
    scales uint8 [N, K/32] (K a multiple of 32).  For a gated product the
    first half of the rows is the gate, the second the up projection."""
    codes: torch.Tensor
    scales: torch.Tensor
    K: int

    def __post_init__(self):
        self._check()

    def _check(self):
        _check_codes(self.codes, self.scales)
        if self.K != 32 * self.scales.shape[1]:
            raise ValueError(f"K = {self.K} must be a multiple of 32 and match the scales")

    @property
    def N(self) -> int:
        return self.codes.shape[0]

    @staticmethod
    def quantize(w: torch.Tensor, stream=None) -> "Mxfp4Weight":
        """From a weight matrix [N, K] in bf16, f16 or f32."""
        codes, scales = mxfp4_quantize(w, stream)
        return Mxfp4Weight(codes, scales, w.shape[1])

    def dequantize(self, dtype=torch.float32, stream=None) -> torch.Tensor:
        return mxfp4_dequantize(self.codes, self.scales, self.K, dtype, stream)


def _linear(name, call, size, x, weight, act, stream):
    ld = _rows(x, "x", weight.K)
    if x.dtype not in _DTYPE:
        raise ValueError("x must be bf16 (mxfp4_linear_a4: or f16)")
    if x.device != weight.codes.device:
        raise ValueError("x and the weight are on different devices")
    T = x.shape[0]
    _int32(name, T, weight.N, weight.K)
    weight._check()   # as it is now: its arrays' memory may have been exchanged since
    c = _byref(dc.mxfp4_weight(weight.codes.data_ptr(), weight.scales.data_ptr(), weight.N, weight.K))
    with _on(stream, x, weight.codes, weight.scales):
        y = x.new_empty((T, weight.N // 2 if act else weight.N))
        need = size(T, c, act)
        ws = _bytes(need, x) if need > 256 else None   # few tokens take none
        check(call(x.data_ptr(), _DTYPE[x.dtype], ld, T, c, act, y.data_ptr(), None if ws is None else ws.data_ptr(),
                   need, _raw_stream(x.get_device())), name)
    return y


def mxfp4_linear(x: torch.Tensor, weight: Mxfp4Weight, activation: str | None = None, stream=None) -> torch.Tensor:
    """W4A16: y [T, N] = x weight^T for bf16 x [T, K]; with an activation the
    gated form y [T, N/2] = act(x Wg^T) * (x Wu^T).  Not differentiable: a backward
    pass through y raises."""
    act = _act(activation)
    if stream is None:
        y = _calls.linear(x, weight.codes, weight.scales, act, False)
        if y is not None:
            return y
    if _recorded(x):
        return _Undifferentiated.apply(lambda: mxfp4_linear(x, weight, activation, stream),
                                       "mxfp4_linear has no backward pass: give it x.detach()", x)
    return _linear("mxfp4_linear", dc.mxfp4_linear, dc.mxfp4_linear_workspace_bytes, x, weight, act, stream)


def mxfp4_linear_a4(x: torch.Tensor, weight: Mxfp4Weight, activation: str | None = None, stream=None) -> torch.Tensor:
    """W4A4: mxfp4_linear with x (bf16 or f16) quantised to MXFP4 on the way in."""
    act = _act(activation)
    if stream is None:
        y = _calls.linear(x, weight.codes, weight.scales, act, True)
        if y is not None:
            return y
    if _recorded(x):
        return _Undifferentiated.apply(lambda: mxfp4_linear_a4(x, weight, activation, stream),
                                       "mxfp4_linear_a4 has no backward pass: give it x.detach()", x)
    return _linear("mxfp4_linear_a4", dc.mxfp4_linear_a4, dc.mxfp4_linear_a4_workspace_bytes, x, weight, act, stream)


# ------------------------------------------------------------- feed-forward
def _ffn_weights(gate, up, down, activation) -> dc.gated_ffn_weights:
    act = _act(activation, gated=True)
    if gate.dim() != 2 or gate.shape != up.shape or down.shape != gate.shape[::-1]:
        raise ValueError("weights must be gate, up [I, H] and down [H, I]")
    if not gate.is_cuda:
        raise ValueError("weights must be on a CUDA device")
    _same("gate, up and down", gate, up, down)
    _contiguous("gate, up and down", gate, up, down)
    if gate.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("weights must be bf16 or f16")
    I, H = gate.shape
    _int32("gated_ffn", I, H)
    return dc.gated_ffn_weights(gate.data_ptr(), up.data_ptr(), down.data_ptr(), H, I, act, _DTYPE[gate.dtype])


def gated_ffn_forward(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                      activation: str = "gelu_tanh", save: bool = False, stream=None):
    """y [T, H] = (act(x gate^T) * (x up^T)) down^T, for bf16 or f16 x [T, H],
    gate, up [I, H], down [H, I]; with save, (y, saved) where saved (8 T I bytes and
    padding) is what gated_ffn_backward takes.  The hidden activations are rounded
    to the 16-bit type, but not for a few tokens without save, where y may so
    differ by that rounding.  For autograd there is gated_ffn: a backward pass
    through this y raises, and with save y has no graph, gated_ffn_backward being the
    caller's to call."""
    if stream is None:
        out = _calls.ffn_forward(x, gate, up, down, _act(activation, gated=True), save)
        if out is not None:
            return out
    if not save and _recorded(x, gate, up, down):
        return _Undifferentiated.apply(lambda: gated_ffn_forward(x, gate, up, down, activation, stream=stream),
                                       "gated_ffn_forward has no backward pass of its own: use gated_ffn",
                                       x, gate, up, down)
    f = _ffn_weights(gate, up, down, activation)
    ld = _rows(x, "x", f.H)
    _same("x and the weights", x, gate)
    T = x.shape[0]
    _int32("gated_ffn_forward", T)
    with _on(stream, x, gate, up, down):
        y = x.new_empty((T, f.H))
        if save:
            saved = _bytes(dc.gated_ffn_saved_bytes(T, _byref(f)), x)
            check(dc.gated_ffn_forward(x.data_ptr(), ld, T, _byref(f), y.data_ptr(), saved.data_ptr(), None, 0,
                                       _raw_stream(x.get_device())), "gated_ffn_forward")
            return y, saved
        ws = _bytes(dc.gated_ffn_forward_workspace_bytes(T, _byref(f)), x)
        check(dc.gated_ffn_forward(x.data_ptr(), ld, T, _byref(f), y.data_ptr(), None, ws.data_ptr(), ws.numel(),
                                   _raw_stream(x.get_device())), "gated_ffn_forward")
    return y


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                       saved: torch.Tensor, activation: str = "gelu_tanh", needs=(True, True, True, True),
                       stream=None):
    """(dx, dgate, dup, ddown) of gated_ffn_forward for dy [T, H], given its x
    and saved; None where `needs` is false."""
    if stream is None:
        grads = _calls.ffn_backward(dy, x, gate, up, down, saved, _act(activation, gated=True), *needs)
        if grads is not None:
            return grads
    f = _ffn_weights(gate, up, down, activation)
    ld, lddy = _rows(x, "x", f.H), _rows(dy, "dy", f.H)
    T = x.shape[0]
    _int32("gated_ffn_backward", T)
    _same("dy, x and the weights", dy, x, gate)
    if (dy.shape[0] != T or saved.dtype != torch.uint8 or saved.device != x.device
            or saved.shape != (max(dc.gated_ffn_saved_bytes(T, _byref(f)), 256),)):
        raise ValueError("dy and saved must be those of x's forward pass")
    _contiguous("saved", saved)
    with _on(stream, dy, x, gate, up, down, saved):
        outs = [w.new_empty(w.shape) if need else None for w, need in zip((x, gate, up, down), needs)]
        ws = _bytes(dc.gated_ffn_backward_workspace_bytes(T, _byref(f)), x)
        check(dc.gated_ffn_backward(dy.data_ptr(), lddy, x.data_ptr(), ld, saved.data_ptr(), T, _byref(f),
                                    *(None if o is None else o.data_ptr() for o in outs), ws.data_ptr(), ws.numel(),
                                    _raw_stream(x.get_device())), "gated_ffn_backward")
    return tuple(outs)


def _own_rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy of it, with contiguous rows from a 16-byte boundary."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, down, activation, recorded):
        # needs_input_grad goes by the tensors alone, also where no graph is recorded
        if not recorded or not any(ctx.needs_input_grad[:4]):
            return gated_ffn_forward(x, gate, up, down, activation)
        y, saved = gated_ffn_forward(x, gate, up, down, activation, save=True)
        ctx.save_for_backward(x, gate, up, down, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, gate, up, down, saved = ctx.saved_tensors
        # an expanded gradient (of a sum) has no rows of its own
        grads = gated_ffn_backward(_own_rows(dy), x, gate, up, down, saved, ctx.activation,
                                   ctx.needs_input_grad[:4])
        return (*grads, None, None)


def gated_ffn(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
              activation: str = "gelu_tanh") -> torch.Tensor:
    """gated_ffn_forward as a differentiable torch operation, for x [..., H].
    First derivatives only.  As with every torch operation, a backward pass can
    be captured into a graph only where no earlier autograd graph of the same
    leaves is alive; gated_ffn_forward and gated_ffn_backward have no such limit."""
    y = _GatedFfn.apply(_own_rows(x.reshape(-1, x.shape[-1])), gate, up, down, activation, torch.is_grad_enabled())
    return y.view(x.shape)
