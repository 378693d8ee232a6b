"""The gated block on both sides of the sizes up to which h is kept in two parts."""
import pytest
import torch

import nvfp4_weight_only_router_b200 as lib
from tests import dense_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,I,parts", [(16, 17088, 512, 2), (16, 17096, 512, 1), (9, 30384, 512, 2), (9, 30392, 512, 1)])
def test_hidden_parts(dev, T, H, I, parts, dtype):
    gen = torch.Generator(device=dev).manual_seed(H)

    def rn(*s, k=1.0):
        return (torch.randn(s, generator=gen, device=dev) * k).to(dtype)
    x, gate, up, down = rn(T, H), rn(I, H, k=H ** -0.5), rn(I, H, k=H ** -0.5), rn(H, I, k=I ** -0.5)
    y = lib.gated_ffn_forward(x, gate, up, down)
    ref = R.ffn64(x.double(), gate.double(), up.double(), down.double(), None, "gelu_tanh", dtype, hidden_parts=parts)["y"]
    assert lib.device_status() == 0
    R.assert_within(y, *ref, f"y {T} {H} {I}")
