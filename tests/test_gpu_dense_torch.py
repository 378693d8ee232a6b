"""The dense operators among torch's own modes and objects."""
import pytest
import torch

import nvfp4_weight_only_router_b200 as lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _make(seed, T, H, I, dev, dtype=BF):
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rn(*s, k=1.0):
        return (torch.randn(s, generator=gen, device=dev) * k).to(dtype)
    return rn(T, H), rn(I, H, k=H ** -0.5), rn(I, H, k=H ** -0.5), rn(H, I, k=I ** -0.5)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 40])
def test_gated_ffn_serving_from_parameters(dev, T, mode):
    x, *w = _make(T, T, 352, 160, dev)
    ref = lib.gated_ffn_forward(x, *w)
    params = [torch.nn.Parameter(t) for t in w]
    with mode():
        y = lib.gated_ffn(x, *params)
    assert torch.equal(y, ref) and not y.requires_grad


@pytest.mark.parametrize("T", [1, 40, 600])
def test_weight_arrays_exchanged(dev, T):
    """Arrays that take other memory (set_): products go by the new one."""
    gen = torch.Generator(dev).manual_seed(T)
    x, a, b = (torch.randn(s, generator=gen, device=dev).to(BF) for s in ((T, 96), (64, 96), (64, 96)))
    first, second = lib.Mxfp4Weight.quantize(a), lib.Mxfp4Weight.quantize(b)
    old = first.codes.detach()[:], first.scales.detach()[:]       # keeps the first memory allocated
    for f in (lib.mxfp4_linear, lib.mxfp4_linear_a4):
        ref = f(x, second)
        assert not torch.equal(f(x, first), ref)
    first.codes.set_(second.codes)
    first.scales.set_(second.scales)
    for f in (lib.mxfp4_linear, lib.mxfp4_linear_a4):
        assert torch.equal(f(x, first), f(x, second))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y = f(x, first, stream=s)
        s.synchronize()
        assert torch.equal(y, f(x, second))
    del old


def test_other_threads_run_while_a_launch_waits(dev):
    """Launches into a full queue wait for the GPU; the interpreter goes on."""
    import threading
    import time
    x, *w = _make(3, 4, 64, 64, dev)
    weight = lib.Mxfp4Weight.quantize(w[0])
    lib.mxfp4_linear(x, weight)
    torch.cuda.synchronize()
    gaps, stop = [0.0], threading.Event()

    def other():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.monotonic()
            gaps[0] = max(gaps[0], now - last)
            last = now
    thread = threading.Thread(target=other)
    thread.start()
    # about a second of sleep on the GPU, then more launches than a queue holds
    torch.cuda._sleep(int(1.9e9))
    began = time.monotonic()
    for _ in range(6000):
        lib.mxfp4_linear(x, weight)
    waited = time.monotonic() - began
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    assert lib.device_status() == 0
    assert waited > 0.5, "the queue never filled: the test shows nothing"
    assert gaps[0] < waited / 2, (gaps, waited)


def _forms(dev):
    x, *w = _make(5, 40, 64, 48, dev)
    weight = lib.Mxfp4Weight.quantize(w[0])
    return x, {"linear": lambda t: lib.mxfp4_linear(t, weight), "a4": lambda t: lib.mxfp4_linear_a4(t, weight),
               "quantize": lambda t: lib.mxfp4_quantize(t)[0], "forward": lambda t: lib.gated_ffn_forward(t, *w),
               "ffn": lambda t: lib.gated_ffn(t, *w)}


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("name", ["linear", "a4", "quantize", "forward", "ffn"])
def test_inside_compiled_functions(dev, name):
    """torch.compile leaves the calls as they are (a graph break each)."""
    x, forms = _forms(dev)
    torch._dynamo.reset()

    def f(t):
        return forms[name](t * 2) + 1
    assert torch.equal(torch.compile(f, backend="eager")(x), f(x))


@pytest.mark.parametrize("name", ["linear", "a4", "quantize", "forward", "ffn"])
def test_function_transforms_are_refused(dev, name):
    """Tensors without memory of their own: refused, nothing is launched."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    x, forms = _forms(dev)
    f = forms[name]
    with pytest.raises(RuntimeError):
        torch.func.vmap(f)(torch.stack((x, x)))
    if name != "quantize":
        with pytest.raises(RuntimeError):
            torch.func.grad(lambda t: f(t).float().sum())(x)
    with FakeTensorMode(allow_non_fake_inputs=True) as mode, pytest.raises(RuntimeError):
        f(mode.from_tensor(x))
    assert lib.device_status() == 0


def test_checkpointed_block(dev):
    from torch.utils.checkpoint import checkpoint
    x, *w = _make(6, 40, 64, 48, dev)
    grads = []
    for run in (lambda *t: lib.gated_ffn(*t), lambda *t: checkpoint(lib.gated_ffn, *t, use_reentrant=False)):
        leaves = [t.clone().requires_grad_() for t in (x, *w)]
        run(*leaves).float().sum().backward()
        grads.append([t.grad for t in leaves])
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_lost_gradients_are_refused(dev):
    """An operator without a backward pass: computed as ever, but a backward pass that
    comes to it raises, and so do forward-mode derivatives."""
    import torch.autograd.forward_ad as fw
    x, *w = _make(7, 40, 64, 48, dev)
    weight = lib.Mxfp4Weight.quantize(w[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    forms = [lambda t, **k: lib.mxfp4_linear(t, weight, **k), lambda t, **k: lib.mxfp4_linear_a4(t, weight, "silu", **k),
             lambda t, **k: lib.gated_ffn_forward(t, *w, **k)]
    for f in forms:
        ref = f(x)
        leaf = x.clone().requires_grad_()
        for more in ({}, {"stream": s}):
            y = f(leaf, **more)
            s.synchronize()
            assert torch.equal(y, ref)
            with pytest.raises(RuntimeError, match="has no backward pass"):
                (y.float().sum() + leaf.float().sum()).backward()
        with torch.no_grad():
            y = f(leaf)
            assert torch.equal(y, ref) and not y.requires_grad
        with fw.dual_level():
            assert torch.equal(f(x), ref)
            with pytest.raises(NotImplementedError):
                f(fw.make_dual(x, torch.ones_like(x)))
    for i in range(3):                                    # a weight that requires a gradient
        p = [t.clone().requires_grad_(k == i) for k, t in enumerate(w)]
        with pytest.raises(RuntimeError, match="use gated_ffn"):
            lib.gated_ffn_forward(x, *p).float().sum().backward()
        y, saved = lib.gated_ffn_forward(x, *p, save=True)
        assert not y.requires_grad and lib.gated_ffn_backward(x, x, *p, saved)[i + 1].shape == p[i].shape


def test_threads_call_at_once(dev):
    """Calls of several threads, each on a stream of its own, which the lock no longer
    keeps apart; the first of a process among them."""
    import threading
    sets = [_make(20 + i, (3, 40, 300, 600)[i], 264, 200, dev) for i in range(4)]

    def calls(x, gate, up, down):
        dn = lib.Mxfp4Weight.quantize(down[:, :192].contiguous())
        y, saved = lib.gated_ffn_forward(x, gate, up, down, save=True)
        return (y, *lib.gated_ffn_backward(y, x, gate, up, down, saved), lib.gated_ffn_forward(x, gate, up, down),
                lib.mxfp4_dequantize(*lib.mxfp4_quantize(x), x.shape[1]),
                lib.mxfp4_linear(x[:, :192].contiguous(), dn), lib.mxfp4_linear_a4(x[:, :192].contiguous(), dn))
    torch.cuda.synchronize()
    got = [[] for _ in sets]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(40):
                got[i].append(calls(*sets[i]))
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert lib.device_status() == 0
    for i, s in enumerate(sets):
        ref = calls(*s)
        assert len(got[i]) == 40
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), i
