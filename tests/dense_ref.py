"""Plain 64-bit forms of the dense feed-forward operators, with bounds on how
far 16-bit results computed with fp32 sums may lie from them.

Bounds (all element by element, u = half a step of the 16-bit type relative to
the value: bf16 2^-8, f16 2^-11; f16 also has an absolute step of 2^-24 near
zero, so each of its roundings adds up to 2^-25):
  * a sum of n products in fp32, in any order, each partial result rounded or
    truncated to 24 bits: n 2^-23 sum|a b|;
  * a stored value is rounded once: u |value|;
  * a rounded factor moves a product by u of its magnitude, and a rounded
    argument g of act by |act'| u |g| (|act'| <= 1.13; |act''| <= 1);
  * act is evaluated in fp32 with the fast exponential: 2^-19 relative.
"""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
FAST = 2.0 ** -19


# ------------------------------------------------------------------- MXFP4
def mx_encode(x: np.ndarray):
    """(codes [R, 16 B], scales [R, B]) of float64 x [R, K], by search over the
    grid: nearest value, ties to the even code, the sign kept."""
    R, K = x.shape
    B = -(-K // 32)
    v = np.zeros((R, B * 32))
    v[:, :K] = x
    v = v.reshape(R, B, 32)
    codes, scales = np.zeros((R, B, 32), np.uint8), np.zeros((R, B), np.uint8)
    for r in range(R):
        for b in range(B):
            blk = v[r, b]
            if not np.isfinite(blk).all():
                scales[r, b] = 255
                continue
            top = np.abs(blk).max()
            X = -127 if top == 0 else min(127, max(-127, math.frexp(top)[1] - 1 - 2))
            scales[r, b] = X + 127
            d = np.abs(np.abs(np.ldexp(blk, -X))[:, None] - E2M1[None, :8])
            # nearest; of two equally near, the even code
            order = np.lexsort((np.broadcast_to(np.arange(8) % 2, d.shape), d), axis=1)
            codes[r, b] = order[:, 0] + 8 * np.signbit(blk)
    c = codes.reshape(R, -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).astype(np.uint8), scales


def mx_decode(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    R, B = scales.shape
    c = np.stack((codes & 15, codes >> 4), -1).reshape(R, B, 32)
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
        return (E2M1[c] * s[..., None]).reshape(R, -1)[:, :K]


def mx_round(x: torch.Tensor) -> torch.Tensor:
    """The MXFP4 values of x in float64 (torch, any device): mx_encode's rule
    through comparisons with the midpoints."""
    R, K = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(R, -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    X = (torch.frexp(torch.where(top > 0, top, torch.ones_like(top)))[1] - 3).clamp(-127, 127)
    X = torch.where(top > 0, X, torch.full_like(X, -127)).double()
    a = v.abs() * torch.exp2(-X)
    q = torch.zeros_like(a)
    for lo, hi, even_hi in ((0, .5, 0), (.5, 1, 1), (1, 1.5, 0), (1.5, 2, 1), (2, 3, 0), (3, 4, 1), (4, 6, 0)):
        mid = (lo + hi) / 2
        q = torch.where((a > mid) | ((a == mid) if even_hi else False), torch.full_like(a, hi), q)
    return (torch.copysign(q, v) * torch.exp2(X)).view(R, -1)[:, :K]


# ------------------------------------------------------------- feed-forward
def act64(name: str, g: torch.Tensor) -> torch.Tensor:
    if name == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def act64_grad(name: str, g: torch.Tensor) -> torch.Tensor:
    if name == "silu":
        s = torch.sigmoid(g)
        return s + g * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def dot(a, b):
    """(a b^T, the bound of its fp32 sum's error)."""
    return a @ b.T, a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().T)


def linear64(x, w, act, dtype):
    """(y, bound) of y = x w^T, or of the gated form where act is given."""
    u, tiny = HALF_STEP[dtype], TINY[dtype]
    z, dz = dot(x, w)
    if act is None:
        return z, dz + u * (z.abs() + dz) + tiny
    n = z.shape[1] // 2
    h, dh = gate64(z[:, :n], dz[:, :n], z[:, n:], dz[:, n:], act)
    return h, dh + u * (h.abs() + dh) + tiny


def gate64(g, dg, up, dup, act):
    """(act(g) up, its error bound) for errors dg, dup of the arguments."""
    a = act64(act, g)
    da = 1.13 * dg + FAST * a.abs()
    return a * up, da * up.abs() + (a.abs() + da) * dup + FAST * (a * up).abs()


def ffn64(x, gate, up, down, dy, act, dtype, hidden_parts=1):
    """{name: (value, bound)} of the forward and backward pass; hidden_parts 2: of
    the forward pass with h in two 16-bit parts, the second rounded as a value of
    at most half a step of the first."""
    r, tiny = HALF_STEP[dtype], TINY[dtype]

    def stored(v, e):
        return e + r * (v.abs() + e) + tiny

    g, eg = dot(x, gate)
    u, eu = dot(x, up)
    h, eh = gate64(g, eg, u, eu, act)
    eh = stored(h, eh) if hidden_parts == 1 else eh + r * r * (h.abs() + eh) + tiny
    y, ey = dot(h, down)
    ey = ey * (1 if hidden_parts == 1 else 1 + r)   # the second parts' products
    out = {"y": (y, stored(y, ey + eh @ down.abs().T))}
    if dy is None:
        return out
    # g and u as kept for the backward pass
    sg, su = stored(g, eg), stored(u, eu)
    a, da = act64(act, g), act64_grad(act, g)
    ea, eda = 1.13 * sg + FAST * a.abs(), 1.0 * sg + FAST * (1 + g.abs())
    dh, edh = dot(dy, down.T)
    dg, du = dh * u * da, dh * a
    edg = stored(dg, edh * (u * da).abs() + (dh.abs() + edh) * (su * (da.abs() + eda) + u.abs() * eda))
    edu = stored(du, edh * a.abs() + (dh.abs() + edh) * ea)
    dx0, e0 = dot(dg, gate.T)
    dx1, e1 = dot(du, up.T)
    dx = dx0 + dx1
    out["dx"] = (dx, stored(dx, 2 * (e0 + e1) + edg @ gate.abs() + edu @ up.abs()))
    for name, left, eleft, right, eright in (("dgate", dg, edg, x, None), ("dup", du, edu, x, None),
                                             ("ddown", dy, None, h, eh)):
        v, e = dot(left.T, right.T)
        if eleft is not None:
            e = e + eleft.T @ right.abs()
        if eright is not None:
            e = e + left.abs().T @ eright
        out[name] = (v, stored(v, e))
    return out


def assert_within(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str) -> None:
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    if bad.any():
        i = tuple(int(k) for k in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements out of bound; first at {i}: "
                             f"{got[i].item()!r} for {ref[i].item()!r}, off by {d[i].item():.3e} > {bound[i].item():.3e}")
