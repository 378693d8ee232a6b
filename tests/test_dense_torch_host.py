"""The dense operators' torch side without a GPU: which steps a call takes."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def dense():
    from nvfp4_weight_only_router_b200 import build
    build.build()
    from nvfp4_weight_only_router_b200 import dense
    return dense


@pytest.mark.parametrize("grad,kept", [("off", False), ("inference", False), ("frozen", False), ("on", True)])
def test_gated_ffn_keeps_only_what_a_backward_pass_needs(dense, monkeypatch, grad, kept):
    asked = []

    def forward(x, gate, up, down, activation="gelu_tanh", save=False, stream=None):
        asked.append(save)
        y = torch.zeros_like(x)
        return (y, torch.zeros(256, dtype=torch.uint8)) if save else y
    monkeypatch.setattr(dense, "gated_ffn_forward", forward)
    x = torch.zeros(2, 3, 16, dtype=torch.bfloat16)
    w = [torch.nn.Parameter(torch.zeros(s, dtype=torch.bfloat16), requires_grad=grad != "frozen")
         for s in ((8, 16), (8, 16), (16, 8))]
    mode = {"off": torch.no_grad, "inference": torch.inference_mode}.get(grad, torch.enable_grad)
    with mode():
        y = dense.gated_ffn(x, *w)
    assert asked == [kept] and y.requires_grad == kept and y.shape == x.shape


@pytest.mark.parametrize("a4", [False, True])
def test_products_read_the_arrays_that_a_weight_has_now(dense, monkeypatch, a4):
    """Memory exchanged under a weight (set_, resize_) leaves no old address in use."""
    monkeypatch.setattr(dense, "_check_codes", lambda *t: None)
    seen = []

    def linear(x, *args):
        seen.append(args)
        return x
    monkeypatch.setattr(dense, "_calls", type("Calls", (), {"linear": staticmethod(linear)}))
    weight = dense.Mxfp4Weight(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), 64)
    codes = torch.ones(8, 32, dtype=torch.uint8)
    weight.codes.set_(codes)
    (dense.mxfp4_linear_a4 if a4 else dense.mxfp4_linear)(torch.zeros(1, 64), weight)
    assert seen[0][0].data_ptr() == codes.data_ptr() and seen[0][1].data_ptr() == weight.scales.data_ptr()
    assert seen[0][2:] == (0, a4)


def test_weights_compare_by_identity(dense, monkeypatch):
    monkeypatch.setattr(dense, "_check_codes", lambda *t: None)
    a, b = (dense.Mxfp4Weight(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), 64) for _ in "ab")
    assert a == a and a != b and a in [b, a] and len({a, b, a}) == 2


@pytest.mark.parametrize("which", ["linear T", "linear N", "linear_a4 T", "linear_a4 N", "forward", "forward save", "backward",
                                   "weights H"])
def test_sizes_past_32_bits_are_refused(dense, monkeypatch, which):
    """They would reach the C call cut to their low 32 bits."""
    import contextlib
    from nvfp4_weight_only_router_b200 import capi
    for name in ("_check_codes", "_same", "_contiguous"):
        monkeypatch.setattr(dense, name, lambda *t: None)
    monkeypatch.setattr(dense, "_rows", lambda t, *a: t.shape[1])
    monkeypatch.setattr(dense, "_on", lambda *t: contextlib.nullcontext())
    monkeypatch.setattr(dense, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(dense, "_calls", type("Calls", (), {n: staticmethod(lambda *a: None)
                                                            for n in ("linear", "ffn_forward", "ffn_backward")}))

    class Weights(torch.Tensor):
        is_cuda = True

    def meta(*s, dtype=torch.bfloat16):
        return torch.Tensor._make_subclass(Weights, torch.empty(s, dtype=dtype, device="meta"))
    big = 2 ** 32 + 8
    with pytest.raises(capi.NVFP4Error) as e:
        if which.startswith("linear"):
            N, T = (big, 4) if which.endswith("N") else (8, big)
            w = dense.Mxfp4Weight(meta(N, 16, dtype=torch.uint8), meta(N, 1, dtype=torch.uint8), 32)
            getattr(dense, "mxfp4_" + which.split()[0])(meta(T, 32), w)
        else:
            H, T = (big, 4) if which == "weights H" else (16, big)
            gate, up, down, x = meta(8, H), meta(8, H), meta(H, 8), meta(T, H)
            if which == "backward":
                dense.gated_ffn_backward(x, x, gate, up, down, meta(1 << 40, dtype=torch.uint8))
            else:
                dense.gated_ffn_forward(x, gate, up, down, save=which.endswith("save"))
    assert e.value.status == capi.NVFP4_ERR_UNSUPPORTED


def test_gradients_are_not_lost_in_silence(dense, monkeypatch):
    """Operators without a backward pass raise where one comes to them, and answer as
    before where none is recorded."""
    monkeypatch.setattr(dense, "_check_codes", lambda *t: None)
    monkeypatch.setattr(dense, "_calls", type("Calls", (), {
        # as the C++ step: nothing where autograd follows
        "linear": staticmethod(lambda x, *a: None if dense._recorded(x) else x.detach() + 1), "ffn_forward": staticmethod(
            lambda x, *a: (x.detach() + 1, torch.zeros(1)) if a[-1] else
            None if dense._recorded(x, *a[:3]) else x.detach() + 1)}))
    weight = dense.Mxfp4Weight(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), 64)
    x, w = torch.zeros(2, 64), torch.zeros(8, 64)
    calls = {"mxfp4_linear ": lambda x: dense.mxfp4_linear(x, weight), "mxfp4_linear_a4": lambda x: dense.mxfp4_linear_a4(x, weight),
             "gated_ffn": lambda x: dense.gated_ffn_forward(x, w, w, w.T)}
    for text, call in calls.items():
        leaf = x.clone().requires_grad_()
        y = call(leaf)
        assert torch.equal(y, x + 1)
        y += 1                                   # not a view: may be changed in place
        with pytest.raises(RuntimeError, match=text):
            (y.sum() + leaf.sum()).backward()
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                assert not call(leaf).requires_grad
        assert not call(x).requires_grad
    p = torch.nn.Parameter(w)
    with pytest.raises(RuntimeError, match="use gated_ffn"):
        dense.gated_ffn_forward(x, p, w, w.T).sum().backward()
    y, _ = dense.gated_ffn_forward(x, p, w, w.T, save=True)
    assert not y.requires_grad


@pytest.mark.parametrize("moe,other,answers", [(0, 0, [0, 0]), (5, 0, [5, 0]), (0, 5, [5, 0]), (7, 5, [7, 5, 0])])
def test_device_status_loses_neither_librarys_error(dense, monkeypatch, moe, other, answers):
    import nvfp4_weight_only_router_b200 as lib
    from nvfp4_weight_only_router_b200 import api, capi, dense_capi
    words = {"moe": moe, "dense": other}

    monkeypatch.setattr(api, "_stream", lambda s=None: 0)
    monkeypatch.setattr(capi, "nvfp4_get_device_status", lambda s: _take(words, "moe"))
    monkeypatch.setattr(dense_capi, "nvfp4dense_get_device_status", lambda s: _take(words, "dense"))
    assert [lib.device_status() for _ in answers] == answers


def _take(words, which):
    got, words[which] = words[which], 0
    return got


def test_device_status_without_the_dense_library():
    """Where the dense library was never loaded no kernel of it has run: its word is
    not asked for, and the library need not be there."""
    import subprocess
    import sys
    code = ("import sys\n"
            "from nvfp4_weight_only_router_b200 import api, capi\n"
            "sys.modules['nvfp4_weight_only_router_b200.dense_capi'] = None\n"      # its import fails
            "api._stream = lambda s=None: 0\n"
            "capi.nvfp4_get_device_status = lambda s: 3\n"
            "assert api.device_status() == 3\n"
            "capi.nvfp4_get_device_status = lambda s: 0\n"
            "assert api.device_status() == 0\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)


def test_tangents_are_not_lost_in_silence(dense, monkeypatch):
    """Forward-mode derivatives: refused, as gated_ffn refuses them."""
    import torch.autograd.forward_ad as fw
    monkeypatch.setattr(dense, "_check_codes", lambda *t: None)
    step = staticmethod(lambda x, *a: None if dense._recorded(x) else x.clone())   # as the C++ step
    monkeypatch.setattr(dense, "_calls", type("Calls", (), {"linear": step, "ffn_forward": step}))
    weight = dense.Mxfp4Weight(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), 64)
    x, w = torch.zeros(2, 64), torch.zeros(8, 64)
    for call in (lambda x: dense.mxfp4_linear(x, weight), lambda x: dense.mxfp4_linear_a4(x, weight),
                 lambda x: dense.gated_ffn_forward(x, w, w, w.T), lambda x: dense.gated_ffn(x, w, w, w.T)):
        with fw.dual_level():
            assert torch.equal(call(x), x)
            with pytest.raises(NotImplementedError, match="jvp"):
                call(fw.make_dual(x, torch.ones_like(x)))
