"""Cases of the dense feed-forward operators, and their plain forms.

Operators: MXFP4 quantisation (one power-of-two scale per 32 elements, E2M1
codes), the product of 16-bit activations with MXFP4 weights (W4A16), the
product with the activations quantised to MXFP4 as well (W4A4), and the gated
feed-forward block with its backward pass.  Sizes are the layer's (hidden
2816, dense intermediate 2112, stacked gate and up 4224) and ragged ones.
"""
import math

import torch

own = False

OPS = ("quantize", "linear", "linear_a4", "ffn", "ffn_step")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token's activations, quantised on the way into a projection
        {"name": "quantize_token", "op": "quantize", "rows": 1, "K": 2816, "dtype": "bf16"},
        # master weights in fp32 with a ragged last block
        {"name": "quantize_ragged", "op": "quantize", "rows": 1000, "K": 2100, "dtype": "f32"},
        # a stack of expert or dense weight matrices at load time
        {"name": "quantize_stack", "op": "quantize", "rows": 32768, "K": 2816, "dtype": "bf16"},
        # decode of one token: gate and up projections with the gate applied
        {"name": "linear_token", "op": "linear", "T": 1, "N": 4224, "K": 2816, "act": "gelu_tanh"},
        # a decode batch through the down projection
        {"name": "linear_batch", "op": "linear", "T": 64, "N": 2816, "K": 2112, "act": ""},
        # prefill through gate and up
        {"name": "linear_prefill", "op": "linear", "T": 4096, "N": 4224, "K": 2816, "act": "gelu_tanh"},
        # the same three in the W4A4 form; the middle one an odd number of packed tokens
        {"name": "a4_token", "op": "linear_a4", "T": 1, "N": 4224, "K": 2816, "act": "gelu_tanh", "dtype": "bf16"},
        {"name": "a4_odd", "op": "linear_a4", "T": 333, "N": 2816, "K": 2112, "act": "", "dtype": "f16"},
        {"name": "a4_prefill", "op": "linear_a4", "T": 4096, "N": 4224, "K": 2816, "act": "gelu_tanh", "dtype": "bf16"},
        # serving one token in bf16
        {"name": "ffn_token", "op": "ffn", "T": 1, "H": 2816, "I": 2112, "act": "gelu_tanh", "dtype": "bf16"},
        # a training step on a small ragged micro-batch: no size a whole number of tiles
        {"name": "step_ragged", "op": "ffn_step", "T": 1001, "H": 2008, "I": 1000, "act": "silu", "dtype": "f16"},
        # a training step over the block's largest token count
        {"name": "step_large", "op": "ffn_step", "T": 8192, "H": 2816, "I": 2112, "act": "gelu_tanh", "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(OPS)
    if op == "quantize":
        K = log(17, 4096)
        return {"op": op, "rows": min(log(1, 32768), 32768 * 2816 // K), "K": K, "dtype": rng.choice(sorted(TYPES))}
    if op in ("linear", "linear_a4"):
        case = {"op": op, "T": log(1, 4096), "N": 16 * log(8, 264), "K": 32 * log(4, 88),
                "act": rng.choice(("", "gelu_tanh", "silu"))}
        if op == "linear_a4":
            case["dtype"] = rng.choice(("bf16", "f16"))
        return case
    return {"op": op, "T": log(1, 64) if op == "ffn" else log(1, 8192), "H": 8 * log(16, 352), "I": 8 * log(16, 264),
            "act": rng.choice(("gelu_tanh", "silu")), "dtype": rng.choice(("bf16", "f16"))}


# ------------------------------------------------------------------- inputs
def _values(gen, shape, dtype):
    """Activations as a normed residual stream gives them: near normal, with a
    few channels an order of magnitude larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = 1.0 + 15.0 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.01)
    return (x * loud).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        return {**case, "x": _values(gen, (case["rows"], case["K"]), TYPES[case["dtype"]])}
    if op in ("linear", "linear_a4"):
        N, K = case["N"], case["K"]
        x = _values(gen, (case["T"], K), TYPES[case.get("dtype", "bf16")])
        codes, scales = _encode(torch.randn((N, K), generator=gen, device="cuda") / math.sqrt(K))
        state = {**case, "x": x, "codes": _pack(codes), "scales": scales}
        if own:
            import nvfp4_weight_only_router_b200 as lib
            state["weight"] = lib.Mxfp4Weight(state["codes"], state["scales"], K)
        return state
    T, H, I, t = case["T"], case["H"], case["I"], TYPES[case["dtype"]]
    state = {**case, "x": torch.randn((T, H), generator=gen, device="cuda").to(t)}
    for name, shape in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        state[name] = (torch.randn(shape, generator=gen, device="cuda") / math.sqrt(shape[1])).to(t)
    if op == "ffn_step":
        state["dy"] = torch.randn((T, H), generator=gen, device="cuda").to(t)
    return state


# -------------------------------------------------------------- plain forms
def _encode(x):
    """Codes 0..15 [R, ceil(K/32), 32] and E8M0 bytes [R, ceil(K/32)] of x;
    in 64 bits, where the scaled values are exact next to the grid's borders."""
    R, K = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(R, -1, 32)
    amax = v.abs().amax(-1)
    finite = torch.isfinite(v).all(-1)
    e = torch.frexp(torch.where(finite & (amax > 0), amax, torch.ones_like(amax)))[1] - 3  # floor(log2) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    scales = torch.where(finite, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    v = torch.where(finite[..., None], v, torch.zeros_like(v)) * torch.exp2(-e.double())[..., None]
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + 8 * torch.signbit(v)).to(torch.uint8), scales


def _pack(codes):
    c = codes.reshape(codes.shape[0], -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous()


def _grid(device):
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=device)


def _decode(codes, scales):
    """fp32 values [R, blocks 32] of codes [R, blocks, 32]."""
    e = scales.int() - 127
    p = torch.where(scales == 255, torch.full_like(scales, float("nan"), dtype=torch.float32), torch.exp2(e.float()))
    return (_grid(codes.device)[codes.int()] * p[..., None]).flatten(1)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1, 32)


def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        codes, scales = _encode(s["x"])
        return {"values": _decode(codes, scales)[:, :s["K"]], "scales": scales}
    if op in ("linear", "linear_a4"):
        x = s["x"]
        a = x.float() if op == "linear" else _decode(*_encode(x))
        z = a @ _decode(_unpack(s["codes"]), s["scales"]).T
        if s["act"]:
            g, u = z.chunk(2, 1)
            z = _act(s["act"], g) * u
        return z.to(x.dtype)
    t = s["x"].dtype
    x, gate, up, down = (s[k].float() for k in ("x", "gate", "up", "down"))
    g, u = x @ gate.T, x @ up.T
    a = _act(s["act"], g)
    h = a * u
    y = (h @ down.T).to(t)
    if op == "ffn":
        return y
    dy = s["dy"].float()
    dh = dy @ down
    dg, du = dh * u * _act_grad(s["act"], g), dh * a
    return {"y": y, "dx": (dg @ gate + du @ up).to(t), "dgate": (dg.T @ x).to(t), "dup": (du.T @ x).to(t),
            "ddown": (dy.T @ h).to(t)}


def _own(s):
    import nvfp4_weight_only_router_b200 as lib
    op = s["op"]
    if op == "quantize":
        codes, scales = lib.mxfp4_quantize(s["x"])
        return {"values": lib.mxfp4_dequantize(codes, scales, s["K"]), "scales": scales}
    if op == "linear":
        return lib.mxfp4_linear(s["x"], s["weight"], activation=s["act"] or None)
    if op == "linear_a4":
        return lib.mxfp4_linear_a4(s["x"], s["weight"], activation=s["act"] or None)
    w = (s["gate"], s["up"], s["down"])
    if op == "ffn":
        return lib.gated_ffn_forward(s["x"], *w, activation=s["act"])
    y, saved = lib.gated_ffn_forward(s["x"], *w, activation=s["act"], save=True)
    dx, dgate, dup, ddown = lib.gated_ffn_backward(s["dy"], s["x"], *w, saved, activation=s["act"])
    return {"y": y, "dx": dx, "dgate": dgate, "dup": dup, "ddown": ddown}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "quantize":
        R, K = case["rows"], case["K"]
        nb = -(-K // 32)
        # the values come back as fp32, and the scales
        return {"bytes": R * K * TYPES[case["dtype"]].itemsize + R * (4 * K + nb), "flops": 2 * R * K}
    if op in ("linear", "linear_a4"):
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": 2 * T * K + N * K * 17 // 32 + 2 * T * (N // 2 if case["act"] else N), "flops": 2 * T * N * K}
    T, H, I = case["T"], case["H"], case["I"]
    if op == "ffn":
        return {"bytes": 2 * (2 * T * H + 3 * I * H), "flops": 6 * T * H * I}
    # x, dy, the weights in; y, dx and the weights' gradients out
    return {"bytes": 2 * (4 * T * H + 6 * I * H), "flops": 18 * T * H * I}


# -------------------------------------------------------------------- exact
def _quantised64(x):
    """The values that MXFP4 keeps of x, in 64 bits: nearest point of the grid
    2^X {0, .5, 1, 1.5, 2, 3, 4, 6} by distance, ties to the even code."""
    R, K = x.shape
    nb = -(-K // 32)
    v = torch.zeros((R, nb * 32), dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    v = v.view(R, nb, 32)
    top = v.abs().max(-1).values
    X = torch.floor(torch.log2(top))
    X = torch.where(torch.exp2(X) > top, X - 1, X)
    X = torch.where(torch.exp2(X + 1) <= top, X + 1, X)
    X = torch.where(top == 0, torch.full_like(X, -127.0), X - 2).clamp(-127, 127)
    w = v.abs() / torch.exp2(X)[..., None]
    best, dist = torch.zeros_like(w), w.clone()
    for code, p in enumerate((0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), 1):
        d = (w - p).abs()
        nearer = (d < dist) | ((d == dist) & (code % 2 == 0))
        best, dist = torch.where(nearer, torch.full_like(best, p), best), torch.where(nearer, d, dist)
    return (torch.copysign(best, v) * torch.exp2(X)[..., None]).view(R, -1)[:, :K], (X + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        values, scales = _quantised64(s["x"])
        return {"values": values, "scales": scales}
    if op in ("linear", "linear_a4"):
        a = s["x"].double() if op == "linear" else _quantised64(s["x"])[0]
        lo, hi = (s["codes"] % 16).long(), (s["codes"] // 16).long()
        mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
        w = torch.empty((s["N"], s["K"]), dtype=torch.float64, device="cuda")
        w[:, 0::2] = mag[lo % 8] * (1 - 2 * (lo // 8))
        w[:, 1::2] = mag[hi % 8] * (1 - 2 * (hi // 8))
        w *= torch.pow(2.0, s["scales"].double() - 127).repeat_interleave(32, 1)
        z = torch.einsum("tk,nk->tn", a, w)
        if s["act"]:
            half = s["N"] // 2
            g, u = z[:, :half], z[:, half:]
            z = (g * torch.sigmoid(g) if s["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")) * u
        return z
    x, gate, up, down = (s[k].double().requires_grad_(op == "ffn_step") for k in ("x", "gate", "up", "down"))
    g, u = torch.einsum("th,ih->ti", x, gate), torch.einsum("th,ih->ti", x, up)
    a = g * torch.sigmoid(g) if s["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    y = torch.einsum("ti,hi->th", a * u, down)
    if op == "ffn":
        return y
    dx, dgate, dup, ddown = torch.autograd.grad(y, (x, gate, up, down), s["dy"].double())
    return {"y": y.detach(), "dx": dx, "dgate": dgate, "dup": dup, "ddown": ddown}
