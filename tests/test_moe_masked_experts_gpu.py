"""A bias of minus infinity masks an expert whatever its products are: rows of the
router that are padding may hold anything, and a token's NaN or infinity must not bring
a masked expert back.  The reference routes over the experts that are left."""
import numpy as np
import pytest
import torch

import block_wise_bit_amd as dq4
from moe_cases import TYPES, route64, to64

pytestmark = pytest.mark.gpu


def coarse(rng, shape, dt):
    """Multiples of 2^-6 below 4: sums of products are exact in 64 bits."""
    return torch.from_numpy(rng.integers(-200, 201, shape) / 64.0).to(TYPES[dt][0])


def masked_checked(x, router, top_k, bias, renormalize):
    ids, weights = dq4.dq4_moe_route(x.cuda(), router.cuda(), top_k, bias=torch.from_numpy(bias).cuda(),
                                     renormalize=renormalize)
    keep = np.flatnonzero(bias != -np.inf)
    with np.errstate(invalid="ignore"):
        left, w, bound = route64(x, router[torch.from_numpy(keep)], min(top_k, keep.size), bias[keep], renormalize)
    want, share, off = np.full((x.shape[0], top_k), -1), np.zeros((x.shape[0], top_k)), np.full((x.shape[0], top_k), 2.0 ** -125)
    want[:, :left.shape[1]] = np.where(left >= 0, keep[left], -1)
    share[:, :left.shape[1]] = w
    off[:, :left.shape[1]] = np.where(np.isfinite(bound), bound, 2.0 ** -125)  # (no place: exactly 0)
    assert np.array_equal(ids.cpu().numpy(), want)
    got = to64(weights)
    assert np.array_equal(np.isnan(got), np.isnan(share))
    nan = np.isnan(share)
    assert (np.abs(np.where(nan, 0, got - share)) <= np.where(nan, 0, off)).all()
    return ids, weights


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("m,E,k,n", [(1, 8, 2, 64), (4, 9, 5, 33), (16, 64, 8, 512), (600, 12, 4, 40)])
def test_rows_of_masked_experts_are_not_looked_at(dt, renormalize, m, E, k, n):
    rng = np.random.default_rng(m + E)
    x, router = coarse(rng, (m, n), dt), coarse(rng, (E, n), dt)
    bias = rng.integers(-50, 51, E).astype(np.float32) / 16
    masked = rng.permutation(E)[:E - max(1, k - 1)]  # fewer are left than are asked for
    bias[masked] = -np.inf
    clean = masked_checked(x, router, k, bias, renormalize)
    for value in (float("nan"), float("inf"), float("-inf")):
        dirty = router.clone()
        dirty[torch.from_numpy(masked)] = value
        got = masked_checked(x, dirty, k, bias, renormalize)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("m,E", [(3, 10), (700, 10)])
def test_a_token_that_is_not_finite_does_not_choose_masked_experts(value, m, E):
    rng = np.random.default_rng(E)
    x, router = coarse(rng, (m, 48), "bf16"), coarse(rng, (E, 48), "bf16")
    x[1, 7] = value
    router[:, 7] = torch.where(router[:, 7] == 0, torch.ones(()).bfloat16(), router[:, 7])
    bias = np.zeros(E, np.float32)
    bias[[0, 1, 4]] = -np.inf
    ids, _ = masked_checked(x, router, 8, bias, True)
    assert not bool(((ids == 0) | (ids == 1) | (ids == 4)).any())
    ids, weights = masked_checked(x, router, 3, np.full(E, -np.inf, np.float32), False)
    assert bool((ids == -1).all()) and bool((weights == 0).all())
