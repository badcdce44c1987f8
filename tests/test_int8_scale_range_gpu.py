"""The 8-bit product under scales of any size: a token's and a channel's scale whose
product is ordinary, while each of them is next to an end of FP32's range.  The bound
is int8_cases.py's: five roundings of FP32, whatever the scales, and the rounding to T."""
import numpy as np
import pytest
import torch

import block_wise_bit_amd as dq4
from int8_cases import TYPES, check, linear64, to64

pytestmark = pytest.mark.gpu

# (channel, token): their product times up to k and times down to 1 / 127^2 stays well
# inside BF16; the last pairs have a subnormal scale
SCALES = [(1e34, 1e-20), (1e-20, 1e34), (2e38, 2e-38), (2e-38, 2e38), (1e36, 1e-38), (1e-38, 1e36), (1e-42, 1e36),
          (1e36, 1e-42), (1.0, 1.0)]


def inputs(m, n, k, w, s, largest, seed):
    rng = np.random.default_rng(seed)
    if largest:  # sums of 127^2 k
        codes, CB = np.full((m, k), 127, np.int8), np.full((n, k), 127, np.int8)
        CB[1::2] = -127
    else:        # sums of 0 and of +-1: one place a row
        codes, CB = np.zeros((m, k), np.int8), rng.integers(-1, 2, (n, k), dtype=np.int8)
        codes[np.arange(m), rng.integers(0, k, m)] = 1
    SCB = torch.from_numpy((w * (0.5 + rng.random(n) / 2)).astype(np.float32))
    scales = (s * (0.5 + rng.random(m) / 2)).astype(np.float32)
    return torch.from_numpy(codes), torch.from_numpy(scales), torch.from_numpy(CB), SCB


@pytest.mark.parametrize("largest", [True, False])
@pytest.mark.parametrize("w,s", SCALES)
@pytest.mark.parametrize("m,n,k", [(1, 40, 64), (5, 33, 100), (20, 64, 4096), (40, 100, 256), (80, 129, 64),
                                   (70, 200, 4112), (300, 260, 640)])
def test_scales_at_the_ends_of_the_range(m, n, k, w, s, largest):
    codes, scales, CB, SCB = inputs(m, n, k, w, s, largest, m + n)
    assert bool((scales > 0).all()) and bool((SCB > 0).all()) and bool(torch.isfinite(SCB).all())
    y = dq4.dq4_int8_linear(codes.cuda(), scales.cuda(), CB.cuda(), SCB.cuda(), dtype=torch.bfloat16)
    want, bound = linear64("bf16", codes.numpy(), scales.numpy().astype(np.float64), CB, SCB)
    check(y, want, bound, f"{m}x{n}x{k} {w} {s}")


@pytest.mark.parametrize("m", [3, 90])
def test_values_beyond_the_type_and_special_scales(m):
    """Infinite, zero and NaN scales keep their meaning, and a value beyond T is an
    infinity."""
    n, k = 6, 64
    codes, CB = torch.ones((m, k), dtype=torch.int8), torch.ones((n, k), dtype=torch.int8)
    SCB = torch.tensor([1.0, 0.0, float("inf"), float("nan"), 3e38, 1e-45])
    scales = torch.ones(m)
    scales[1], scales[2] = 0.0, float("nan")
    y = to64(dq4.dq4_int8_linear(codes.cuda(), scales.cuda(), CB.cuda(), SCB.cuda(), dtype=torch.float16))
    one = 64 / 16129.0
    for t in range(m):
        if t == 2:
            assert np.isnan(y[t]).all()
            continue
        assert np.isnan(y[t, 3]) and y[t, 1] == 0 and y[t, 5] == 0
        if t == 1:
            assert y[t, 0] == 0 and y[t, 4] == 0 and np.isnan(y[t, 2])
        else:
            assert abs(y[t, 0] - one) <= one * (2.0 ** -11 + 2.0 ** -20) and y[t, 2] == np.inf and y[t, 4] == np.inf
