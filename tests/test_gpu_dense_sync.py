"""Short launches of the two-SM kernel one after the other: pairs that leave while
the next launch waits to take their shared memory, in every form."""
import pytest
import torch

import nvfp4_weight_only_router_b200 as lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [(33, 304, 32), (129, 2368, 64), (130, 1184, 160), (2100, 304, 96)])
def test_short_launches_in_a_row(dev, T, N, K):
    gen = torch.Generator(dev).manual_seed(T)

    def rn(*s, k=1.0):
        return (torch.randn(s, generator=gen, device=dev) * k).bfloat16()
    weight = lib.Mxfp4Weight.quantize(rn(N, K))
    gate, up, down, dy = rn(N, K, k=K ** -0.5), rn(N, K, k=K ** -0.5), rn(K, N, k=N ** -0.5), rn(T, K)
    xs = [rn(T, K) for _ in range(3)]

    def calls(x):
        y, saved = lib.gated_ffn_forward(x, gate, up, down, "silu", save=True)
        return (lib.mxfp4_linear(x, weight), lib.mxfp4_linear(x, weight, "silu"), lib.mxfp4_linear_a4(x, weight),
                lib.mxfp4_linear_a4(x, weight, "silu"), y, *lib.gated_ffn_backward(dy, x, gate, up, down, saved, "silu"))
    ref = []
    for x in xs:
        one = []
        for t in calls(x):
            torch.cuda.synchronize()
            one.append(t)
        ref.append(one)
    got = [calls(xs[i % 3]) for i in range(60)]
    torch.cuda.synchronize()
    assert lib.device_status() == 0
    for i, out in enumerate(got):
        for k, (a, b) in enumerate(zip(out, ref[i % 3])):
            assert torch.equal(a, b), (i, k)
