"""The gated feed-forward block on the GPU, forward and backward, against its
64-bit form (bounds of dense_ref), and the path train -> quantise -> serve."""
import pytest
import torch

import nvfp4_weight_only_router_b200 as lib
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


def _make(seed, T, H, I, dtype, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rn(*s, k=1.0):
        return (torch.randn(s, generator=gen, device=dev) * k).to(dtype)
    return rn(T, H), rn(I, H, k=H ** -0.5), rn(I, H, k=H ** -0.5), rn(H, I, k=I ** -0.5), rn(T, H)


def _reference(x, gate, up, down, dy, act):
    return R.ffn64(x.double(), gate.double(), up.double(), down.double(), None if dy is None else dy.double(), act,
                   x.dtype)


def _check_step(x, gate, up, down, dy, act):
    y, saved = lib.gated_ffn_forward(x, gate, up, down, act, save=True)
    grads = lib.gated_ffn_backward(dy, x, gate, up, down, saved, act)
    ref = _reference(x, gate, up, down, dy, act)
    assert lib.device_status() == 0
    for name, got in zip(("y", "dx", "dgate", "dup", "ddown"), (y, *grads)):
        R.assert_within(got, *ref[name], f"{name} {list(x.shape)} {list(gate.shape)} {act} {x.dtype}")
    return y, saved, grads


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,H,I", [(1, 64, 64), (7, 8, 8), (9, 72, 136), (32, 256, 200), (33, 256, 200), (100, 520, 264),
                                   (129, 128, 1000), (255, 640, 64), (300, 2816, 704), (1, 4000, 72), (6, 5000, 3400),
                                   (13, 4000, 72), (25, 2832, 3000), (60, 4000, 72), (100, 2000, 6000)])
def test_forward(dev, T, H, I, dtype):
    x, gate, up, down, _ = _make(T, T, H, I, dtype, dev)
    for act in ("gelu_tanh", "silu"):
        y = lib.gated_ffn_forward(x, gate, up, down, act)
        assert lib.device_status() == 0
        R.assert_within(y, *_reference(x, gate, up, down, None, act)["y"], f"y {T} {H} {I} {act}")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,H,I", [(T, H, I) for T in (1, 2, 3, 4) for H, I in ((352, 160), (8, 8), (136, 4000), (2816, 2112))]
                                  + [(5, 8, 8), (8, 352, 160), (9, 136, 512), (16, 2816, 512)])
def test_few_tokens_round_once(dev, T, H, I, dtype):
    """For few tokens y is off by its own rounding, not by that of h as well."""
    x, gate, up, down, _ = _make(T + I, T, H, I, dtype, dev)
    for act, k in (("gelu_tanh", 1.0), ("silu", 1.0), ("silu", 2.0 ** -7)):   # k: h among f16's smallest numbers
        z = x * k
        y = lib.gated_ffn_forward(z, gate, up, down, act)
        ref = R.ffn64(z.double(), gate.double(), up.double(), down.double(), None, act, dtype, hidden_parts=2)["y"]
        assert lib.device_status() == 0
        R.assert_within(y, *ref, f"y {T} {H} {I} {act} {k}")


@pytest.mark.parametrize("T", [3, 10])
def test_few_tokens_beyond_f16(dev, T):
    """An h past f16's range is the infinity that it is with more tokens, and
    reaches its token alone."""
    x, gate, up, down, _ = _make(5, T, 64, 48, F16, dev)
    clean = lib.gated_ffn_forward(x, gate, up, down)
    x[1] *= 3000
    y = lib.gated_ffn_forward(x, gate, up, down)
    many = lib.gated_ffn_forward(x.repeat(20, 1), gate, up, down)[:T]
    assert torch.equal(y[0], clean[0]) and torch.equal(y[2:], clean[2:])
    assert not torch.isfinite(many[1]).all()
    assert torch.equal(torch.isnan(y[1]), torch.isnan(many[1])) and torch.equal(torch.isinf(y[1]), torch.isinf(many[1]))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,H,I", [(1, 64, 64), (5, 8, 8), (31, 72, 136), (64, 256, 256), (65, 264, 200), (130, 520, 264),
                                   (257, 128, 1000), (1000, 640, 64), (513, 1024, 768)])
def test_step(dev, T, H, I, dtype):
    for act in ("gelu_tanh", "silu"):
        _check_step(*_make(T + I, T, H, I, dtype, dev), act)


@pytest.mark.parametrize("T,H,I,act,dtype", [(1001, 2008, 1000, "silu", F16), (4096, 2816, 2112, "gelu_tanh", BF)])
def test_step_large(dev, T, H, I, act, dtype):
    _check_step(*_make(3, T, H, I, dtype, dev), act)


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_large_gates(dev, act):
    """Gate values far outside the activation's curved range: finite gradients."""
    x, gate, up, down, dy = _make(5, 40, 64, 64, BF, dev)
    gate = gate * 64
    _check_step(x, gate, up, down, dy, act)


def test_partial_gradients_and_empty_batch(dev):
    x, gate, up, down, dy = _make(6, 70, 136, 72, BF, dev)
    y, saved, full = _check_step(x, gate, up, down, dy, "gelu_tanh")
    for needs in ((True, False, False, False), (False, True, False, True), (False, False, False, True),
                  (False, False, True, False), (False,) * 4):
        part = lib.gated_ffn_backward(dy, x, gate, up, down, saved, needs=needs)
        for p, f, n in zip(part, full, needs):
            assert (p is None) if not n else torch.equal(p, f)
    y0, s0 = lib.gated_ffn_forward(x[:0], gate, up, down, save=True)
    g0 = lib.gated_ffn_backward(dy[:0], x[:0], gate, up, down, s0)
    assert y0.shape == (0, 136) and g0[0].shape == (0, 136)
    assert all((g == 0).all() for g in g0[1:])
    assert lib.gated_ffn_forward(x[:0], gate, up, down).shape == (0, 136)


@pytest.mark.parametrize("T", [4, 90])
def test_strides_streams_and_graphs(dev, T):
    x, gate, up, down, dy = _make(7, T, 136, 72, BF, dev)
    wide = torch.zeros((T, 400), dtype=BF, device=dev)
    wide[:, 8:144], wide[:, 200:336] = x, dy
    xs, ds = wide[:, 8:144], wide[:, 200:336]
    y, saved = lib.gated_ffn_forward(x, gate, up, down, save=True)
    grads = lib.gated_ffn_backward(dy, x, gate, up, down, saved)
    serve = lib.gated_ffn_forward(x, gate, up, down)

    def same(a, b):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    ys, ss = lib.gated_ffn_forward(xs, gate, up, down, save=True)
    same((ys, *lib.gated_ffn_backward(ds, xs, gate, up, down, ss)), (y, *grads))
    same((lib.gated_ffn_forward(xs, gate, up, down),), (serve,))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, s2 = lib.gated_ffn_forward(x, gate, up, down, save=True, stream=s)
    g2 = lib.gated_ffn_backward(dy, x, gate, up, down, s2, stream=s)
    s.synchronize()
    same((y2, *g2), (y, *grads))
    # two captured graphs and eager calls between their replays
    static, outs, graphs = x.clone(), [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            yc, sc = lib.gated_ffn_forward(static, gate, up, down, save=True)
            outs.append((yc, *lib.gated_ffn_backward(dy, static, gate, up, down, sc),
                         lib.gated_ffn_forward(static, gate, up, down)))
        graphs.append(g)
    static.copy_(x.flip(0))
    for g in graphs:
        g.replay()
    lib.gated_ffn_forward(x, gate, up, down)
    yf, sf = lib.gated_ffn_forward(x.flip(0), gate, up, down, save=True)
    ref = (yf, *lib.gated_ffn_backward(dy, x.flip(0), gate, up, down, sf), lib.gated_ffn_forward(x.flip(0), gate, up, down))
    torch.cuda.synchronize()
    for o in outs:
        same(o, ref)


def test_autograd(dev):
    x, gate, up, down, _ = _make(8, 60, 136, 72, BF, dev)
    leaves = [t.clone().requires_grad_() for t in (x.view(3, 20, 136), gate, up, down)]
    y = lib.gated_ffn(*leaves, "silu")
    assert y.shape == (3, 20, 136)
    y.sum().backward()                       # an expanded gradient
    yf, saved = lib.gated_ffn_forward(x, gate, up, down, "silu", save=True)
    ref = lib.gated_ffn_backward(torch.ones_like(x), x, gate, up, down, saved, "silu")
    assert torch.equal(y.view(60, 136), yf)
    for leaf, g in zip(leaves, ref):
        assert torch.equal(leaf.grad.view(g.shape), g)
    # tokens and an incoming gradient off the 16-byte grid
    flat = torch.empty(1 + x.numel(), dtype=BF, device=dev)
    off = flat[1:].view(60, 136)
    off.copy_(x)
    xo = off.detach().requires_grad_()
    yo = lib.gated_ffn(xo, gate, up, down, "silu")
    go = torch.ones_like(flat)[1:].view(60, 136)
    yo.backward(go)
    assert torch.equal(yo, yf) and torch.equal(xo.grad, ref[0])
    # frozen weights: the input's gradient alone
    xi = x.clone().requires_grad_()
    lib.gated_ffn(xi, gate, up, down, "silu").sum().backward()
    assert torch.equal(xi.grad, ref[0])
    with torch.no_grad():
        assert not lib.gated_ffn(xi, gate, up, down, "silu").requires_grad


def test_shared_weights(dev):
    """One tensor as gate and up: its gradient is the sum of both."""
    x, w, _, down, dy = _make(10, 50, 72, 136, BF, dev)
    leaf = w.clone().requires_grad_()
    lib.gated_ffn(x, leaf, leaf, down).backward(dy)
    y, saved = lib.gated_ffn_forward(x, w, w, down, save=True)
    _, dgate, dup, _ = lib.gated_ffn_backward(dy, x, w, w, down, saved)
    assert torch.equal(leaf.grad, dgate + dup)


def test_refusals(dev):
    x, gate, up, down, dy = _make(11, 40, 64, 48, BF, dev)
    y, saved = lib.gated_ffn_forward(x, gate, up, down, save=True)
    bad = (lambda: lib.gated_ffn_forward(x[:, :32], gate, up, down), lambda: lib.gated_ffn_forward(x.to(F16), gate, up, down),
           lambda: lib.gated_ffn_forward(x, gate, up, down.T), lambda: lib.gated_ffn_forward(x, gate, up[:40], down),
           lambda: lib.gated_ffn_forward(x, gate.T.contiguous().T, up, down), lambda: lib.gated_ffn_forward(x, gate, up, down, None),
           lambda: lib.gated_ffn_forward(x[:1].expand(40, 64), gate, up, down),
           lambda: lib.gated_ffn_forward(x.cpu(), gate, up, down), lambda: lib.gated_ffn_forward(x[0], gate, up, down),
           lambda: lib.gated_ffn_backward(dy[:39], x, gate, up, down, saved),
           lambda: lib.gated_ffn_backward(dy, x, gate, up, down, saved[:-1]),
           lambda: lib.gated_ffn_backward(dy, x, gate, up, down, saved.view(torch.int8)),
           lambda: lib.gated_ffn_backward(dy, x[:33], gate, up, down, saved))
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lib.gated_ffn_forward(x.reshape(-1)[8 * 64 - 60:][:64 * 30].view(30, 64), gate, up, down),  # rows off the grid
                 lambda: lib.gated_ffn_forward(x[:, :60].contiguous(), gate[:, :60].contiguous(), up[:, :60].contiguous(),
                                               down[:60].contiguous())):
        with pytest.raises(lib.NVFP4Error):
            call()
    with pytest.raises(torch.OutOfMemoryError):
        wide = torch.zeros((1 << 18, 8), dtype=BF, device=dev)          # 2 TB to keep
        lib.gated_ffn_forward(torch.zeros((1 << 20, 8), dtype=BF, device=dev), wide, wide, wide.view(8, -1), save=True)
    # nothing was enqueued, and the library still answers
    assert lib.device_status() == 0
    assert torch.equal(lib.gated_ffn_forward(x, gate, up, down, save=True)[0], y)


@pytest.mark.parametrize("T", [3, 200])
def test_train_quantise_serve(dev, T):
    """A step of training in bf16, the stepped weights quantised to MXFP4, and
    the block served from them in both forms."""
    x, gate, up, down, dy = _make(9, T, 256, 192, BF, dev)
    leaves = [t.clone().requires_grad_() for t in (gate, up, down)]
    lib.gated_ffn(x, *leaves).backward(dy)
    gate, up, down = ((t - 0.05 * t.grad).detach() for t in leaves)
    gu, dn = lib.Mxfp4Weight.quantize(torch.cat((gate, up))), lib.Mxfp4Weight.quantize(down)
    for a4, f in ((False, lib.mxfp4_linear), (True, lib.mxfp4_linear_a4)):
        h = f(x, gu, "gelu_tanh")
        y = f(h, dn)
        q = R.mx_round if a4 else torch.Tensor.double
        href, hb = R.linear64(q(x), gu.dequantize().double(), "gelu_tanh", BF)
        R.assert_within(h, href, hb, "h")
        yref, yb = R.linear64(q(h), dn.dequantize().double(), None, BF)   # from the served h
        R.assert_within(y, yref, yb, "y")
    assert lib.device_status() == 0


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_back_to_back_calls(dev, T):
    """Calls in a row overlap at their ends: weights and tokens written by the
    kernel just before, outputs in memory that the call before still reads."""
    sets = [_make(20 + i, T, 256, 192, BF, dev) for i in range(4)]

    def chain(x, gate, up, down):
        gu, dn = lib.Mxfp4Weight.quantize(torch.cat((gate, up))), lib.Mxfp4Weight.quantize(down)
        h = lib.mxfp4_linear(x, gu, "silu")
        y = lib.mxfp4_linear_a4(h, dn)
        z = lib.gated_ffn_forward(y, gate, up, down)                  # h, y and the codes are freed as they are used
        return lib.mxfp4_linear(lib.gated_ffn_forward(z, gate, up, down), gu, "silu")
    ref = []
    for x, gate, up, down, _ in sets:
        ref.append(chain(x, gate, up, down))
        torch.cuda.synchronize()
    xs, gs, us, ds = (torch.empty_like(t) for t in sets[0][:4])
    got = []
    for i in range(60):
        for dst, src in zip((xs, gs, us, ds), sets[i % 4]):
            dst.copy_(src)
        got.append(chain(xs, gs, us, ds))
        lib.mxfp4_dequantize(*lib.mxfp4_quantize(got[-1]))            # its memory is the next call's
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, ref[i % 4]), i


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_fork_and_join(dev, T, captured):
    """Calls that follow copies, memsets, other streams' work and several
    predecessors at once, eager and in a graph."""
    x, gate, up, down, dy = _make(30, T, 256, 192, BF, dev)
    gu = lib.Mxfp4Weight.quantize(torch.cat((gate, up)))
    xin, buf = torch.zeros_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        buf.copy_(xin)                                     # a copy as predecessor
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a = lib.gated_ffn_forward(buf, gate, up, down)
        b = lib.mxfp4_linear_a4(buf, gu, "silu")
        main.wait_stream(side)
        c, saved = lib.gated_ffn_forward(a, gate, up, down, save=True)   # two predecessors
        z = torch.zeros_like(c)
        grads = lib.gated_ffn_backward(z.add_(1), a, gate, up, down, saved)
        q = lib.mxfp4_quantize(b)
        return (a, b, c, *grads, *q, lib.mxfp4_dequantize(*q), lib.mxfp4_linear(a, gu, stream=None))
    xin.copy_(x)
    ref = work()
    torch.cuda.synchronize()
    ref = [t.clone() for t in ref]
    xin.zero_()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = work()
        xin.copy_(x)
        for _ in range(3):
            g.replay()
    else:
        xin.copy_(x)
        for _ in range(3):
            out = work()
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(out, ref))


def test_past_32_bit_offsets(dev):
    """Intermediates of more than 2^31 elements: tokens that are zero but for the
    last, whose outputs and gradients are those of a batch of their own."""
    T, H, I, n = (1 << 20) - 3, 8, 2112, 61
    x, gate, up, down, dy = _make(12, n, H, I, BF, dev)
    xl, dyl = (torch.zeros((T, H), dtype=BF, device=dev) for _ in range(2))
    xl[-n:], dyl[-n:] = x, dy
    y, saved = lib.gated_ffn_forward(xl, gate, up, down, save=True)
    grads = lib.gated_ffn_backward(dyl, xl, gate, up, down, saved)
    ref = _reference(x, gate, up, down, dy, "gelu_tanh")
    assert lib.device_status() == 0
    assert (y[:-n] == 0).all() and (grads[0][:-n] == 0).all()
    for name, got in zip(("y", "dx", "dgate", "dup", "ddown"), (y[-n:], grads[0][-n:], *grads[1:])):
        R.assert_within(got, *ref[name], name)
    R.assert_within(lib.gated_ffn_forward(xl, gate, up, down)[-n:], *ref["y"], "y, not kept")
