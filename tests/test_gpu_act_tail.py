"""The activations' relative error on their negative side, where s = 1 / (1 + exp(-z)) is
small: sums of hidden units of nearly equal size and alternating sign, whose
difference the error of act would swamp if it were larger than stated.

Bound of one h = act(g) u: 2^-20 (1 + 0.6 |z|) of act (in units of 2^-23: the fast
exponential 2 + 1.173 |z|, z's roundings 3.3 |z| (six roundings of half a unit, two of
them of constants), sum, division and product 4: 6 + 4.5 |z| <= 8 + 4.8 |z|), 2^-24 of the product
with u, r^2 of h in two 16-bit parts (r = 2^-11 in f16); the sum of n in fp32 n 2^-23;
y's own rounding."""
import math

import pytest
import torch

import nvfp4_weight_only_router_b200 as lib
from tests import dense_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,lo", [("silu", -9.0), ("gelu_tanh", -3.5)])
def test_negative_gates(dev, act, lo):
    F16, n = torch.float16, 64
    # one feature of the token carries 1: gate, up hold g, u themselves (products with 1, exact)
    g = torch.linspace(lo, -0.75, n, dtype=torch.float64).to(F16).double()
    a = R.act64(act, g)
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64).repeat(n // 2)
    u = (sign / a).to(F16).double()                       # act(g) u = +-(1 + up to 2^-11)
    assert torch.isfinite(u).all()
    x = torch.zeros(1, 8, dtype=F16, device=dev)
    x[0, 0] = 1
    gate, up, down = (torch.zeros(s, dtype=F16, device=dev) for s in ((n, 8), (n, 8), (8, n)))
    gate[:, 0], up[:, 0], down[0] = g.to(dev), u.to(dev), 1
    y = lib.gated_ffn_forward(x, gate, up, down, act)
    assert lib.device_status() == 0
    z = g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    h = a * u
    exact = h.sum()
    bound = (h.abs() * (2.0 ** -20 * (1 + 0.6 * z.abs()) + 2.0 ** -24 + 2.0 ** -22 + n * 2.0 ** -23)).sum()
    bound = bound + 2.0 ** -11 * (exact.abs() + bound) + 2.0 ** -25
    assert bound < 2.0 ** -10                              # far below what 16-bit terms alone would allow (64 x 2^-11)
    assert abs(y[0, 0].double().cpu() - exact) <= bound, (y[0, 0].item(), exact.item(), bound.item())
    assert (y[0, 1:] == 0).all()
