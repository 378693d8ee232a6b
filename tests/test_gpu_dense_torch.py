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
