"""The dense operators' torch side without a GPU: which steps a call takes."""
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
