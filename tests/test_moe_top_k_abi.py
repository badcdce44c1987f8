"""What the calls of include/dq4_moe.h say to more choices a token than there are
experts (no GPU).  The router refuses them.  The experts' call takes them: rows of ids
may hold an expert twice, or ids that are no expert."""
import ctypes

import numpy as np
import pytest

import block_wise_bit_amd as dq4
from libs import ensure_hip_library
from test_linear_abi import weight

P = ctypes.c_void_p
ONE = P(256)


def test_more_choices_than_experts():
    lib = ensure_hip_library()
    for E, k in ((1, 2), (4, 5), (4, 16), (8, 9)):
        for m in (0, 4):
            assert lib.dq4_moe_route(ONE, m, 64, 64, dq4.DQ4_F16, ONE, None, E, k, 1, ONE, ONE, ONE, 1 << 40,
                                     None) == dq4.DQ4_EINVAL, (E, k, m)
        w = ctypes.byref(weight())
        assert lib.dq4_moe_fused(w, w, w, E, 32, 64, dq4.DQ4_F16, dq4.DQ4_ACT_SILU, ONE, 0, 64, ONE, ONE, k, None, 64, ONE,
                                 64, ONE, 1 << 40, None) == dq4.DQ4_OK, (E, k)
        assert lib.dq4_moe_fused_workspace_bytes(E, 32, 64, 4, k) > 0
        assert lib.dq4_moe_route_workspace_bytes(4, E) > 0


def test_header_says_so():
    with open(dq4.MOE_HEADER_PATH) as fh:
        text = " ".join(fh.read().replace("*", " ").split())
    assert "top_k below 1, or above n_experts (dq4_moe_route alone)" in text


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 5, 33])
def test_experts_with_more_choices_than_experts(m):
    import torch
    from moe_cases import Layer, check, moe64
    rng = np.random.default_rng(m)
    E, n_ff, n_in, k = 2, 33, 64, 16
    layer = Layer(E, n_ff, n_in, 32, seed=3)
    ids = rng.integers(-1, E + 1, (m, k)).astype(np.int32)
    weights = rng.random((m, k)).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((m, n_in))).half()
    y = dq4.dq4_moe_fused(*layer.device(), E, n_ff, n_in, 32, x.cuda(), torch.from_numpy(ids).cuda(),
                          torch.from_numpy(weights).cuda())
    check(y, *moe64("f16", "silu", layer, x, ids, weights), f"{k} choices of {E} experts, {m} tokens")
