"""Where the gated block keeps its hidden activations in two 16-bit parts, by the
workspace that it asks for."""
import ctypes

import pytest

P = 4096


@pytest.mark.parametrize("T,H,I,parts", [(4, 1 << 18, 1 << 18, 2), (5, 64, 520, 1), (5, 64, 512, 2), (8, 1 << 18, 512, 2),
                                         (16, 17088, 512, 2), (16, 17096, 512, 1), (9, 1 << 18, 512, 1), (17, 64, 64, 1)])
def test_workspace_holds_the_parts_that_the_call_writes(T, H, I, parts):
    from nvfp4_weight_only_router_b200 import build
    build.build()
    from nvfp4_weight_only_router_b200 import dense_capi as dc
    f = dc.gated_ffn_weights(P, P, P, H, I, 1, 0)
    bytes_ = T * (-(-I // 64) * 64) * 2 * parts
    assert dc.gated_ffn_forward_workspace_bytes(T, ctypes.byref(f)) == -(-(bytes_ + 1) // 256) * 256
