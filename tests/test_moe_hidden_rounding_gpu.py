"""h, the experts' product of act(gate) and up, is rounded to T between the two
products (include/dq4_moe.h): what that costs is pinned on weights that pick single
elements, 0, 1 and -1 as their 4-bit values."""
import pytest
import torch

import block_wise_bit_amd as dq4

pytestmark = pytest.mark.gpu

N = 32  # n_ff and n_in


def picked(entries):
    """A nested 4-bit weight of N x N with the given elements {(row, column): +-1}."""
    codes = torch.zeros(N * N, dtype=torch.uint8)
    for (row, column), sign in entries.items():
        codes[row * N + column] = 1 if sign > 0 else 2
    values = torch.zeros(16)
    values[1], values[2] = 1.0, -1.0
    return dict(packed=(codes[0::2] | codes[1::2] << 4).cuda(), scale_codes=torch.zeros(N, dtype=torch.uint8, device="cuda"),
                nested_absmax=torch.ones(1, device="cuda"), scale_codebook=torch.ones(256, device="cuda"),
                codebook4=values.cuda(), offset=0.0)


def experts(x):
    """y0 = h0 - h1, y1 = h0, h0 = relu(x0) x1, h1 = relu(x2) x3; the rest of y sums zeros."""
    m = x.shape[0]
    return dq4.dq4_moe_fused(picked({(0, 0): 1, (1, 2): 1}), picked({(0, 1): 1, (1, 3): 1}),
                             picked({(0, 0): 1, (0, 1): -1, (1, 0): 1}), 1, N, N, 32, x.cuda(),
                             torch.zeros((m, 1), dtype=torch.int32, device="cuda"), torch.ones((m, 1), device="cuda"),
                             activation="relu").cpu()


@pytest.mark.parametrize("m", [1, 4, 40])
@pytest.mark.parametrize("dt,eps", [(torch.float16, 2.0 ** -10), (torch.bfloat16, 2.0 ** -7)])
def test_h_is_rounded_to_the_type(dt, eps, m):
    x = torch.zeros((m, N), dtype=dt)
    x[:, 0] = x[:, 1] = 1 + eps       # h0 = 1 + 2 eps + eps^2
    x[:, 2], x[:, 3] = 1 + 2 * eps, 1
    y = experts(x)
    assert bool((y[:, 0] == 0).all()) and bool((y[:, 1] == 1 + 2 * eps).all()) and bool((y[:, 2:] == 0).all())


@pytest.mark.parametrize("m", [1, 4, 40])
def test_h_beyond_the_type_is_an_infinity_in_fp16(m):
    x = torch.zeros((m, N), dtype=torch.float16)
    x[:, :4] = 1
    x[m // 2, 0] = x[m // 2, 1] = 300   # h0 = 90000
    y = experts(x)
    assert bool((y[m // 2, :2] == float("inf")).all()) and bool(torch.isnan(y[m // 2, 2:]).all())
    others = [t for t in range(m) if t != m // 2]
    assert bool((y[others, 0] == 0).all()) and bool((y[others, 1] == 1).all())
    y = experts(x.bfloat16())           # BF16 has FP32's range: 90000 rounds to a multiple of 512
    assert y[m // 2, 1] == 176 * 512 and bool(torch.isfinite(y).all())
