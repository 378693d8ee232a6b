"""W4A16 on both sides of the token count above which the weights are decoded once."""
import pytest
import torch

import nvfp4_weight_only_router_b200 as lib
from tests import dense_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("N,K", [(528, 160), (2816, 704)])
@pytest.mark.parametrize("T", [511, 512, 513, 700])
def test_decoded_once_limit(dev, T, N, K, act):
    gen = torch.Generator(dev).manual_seed(T)
    weight = lib.Mxfp4Weight.quantize((torch.randn((N, K), generator=gen, device=dev) * K ** -0.5).bfloat16())
    x = torch.randn((T, K), generator=gen, device=dev).bfloat16()
    y = lib.mxfp4_linear(x, weight, act)
    ref, bound = R.linear64(x.double(), weight.dequantize().double(), act, torch.bfloat16)
    assert lib.device_status() == 0
    R.assert_within(y, ref, bound, f"{T} {N} {K} {act}")
