"""The router on BF16 operands whose products leave FP32's range: the logits are
64-bit sums of exact products.  Inputs are small whole numbers times powers of two,
few to a row, so that every sum is exact in 64 bits in any order."""
import numpy as np
import pytest
import torch

import block_wise_bit_amd as dq4
from moe_cases import to64

pytestmark = pytest.mark.gpu

#: tokens, experts, top_k, row length: a workgroup for a token and an expert, a wave for
#: four experts, rows that take whole vectors and others
SHAPES = [(1, 8, 2, 64), (3, 65, 4, 33), (20, 64, 8, 512), (300, 16, 3, 40), (600, 9, 2, 17)]
PLACES = 5


def operands(m, E, n, exponent, seed):
    """x and the router as (whole number below 128) 2^exponent, in PLACES columns."""
    rng = np.random.default_rng(seed)
    cols = rng.choice(n, PLACES, replace=False)
    x, r = np.zeros((m, n)), np.zeros((E, n))
    x[:, cols] = rng.integers(-127, 128, (m, PLACES)) * 2.0 ** exponent
    r[:, cols] = rng.integers(-127, 128, (E, PLACES)) * 2.0 ** exponent
    r[E // 2] = r[0]  # a tie
    return torch.from_numpy(x).bfloat16(), torch.from_numpy(r).bfloat16()


def checked(x, router, top_k, logits, renormalize):
    """Logits that differ by so much that exp of a difference is 0 or, at a tie, 1 (or,
    `logits` tiny, always 1): a weight is 1 / (the number of ones), off by the reciprocal's
    and the product's last places."""
    ids, weights = dq4.dq4_moe_route(x.cuda(), router.cuda(), top_k, renormalize=renormalize)
    order = np.argsort(-logits, axis=1, kind="stable")
    want = order[:, :top_k]
    assert np.array_equal(ids.cpu().numpy(), want)
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    assert set(np.unique(p)) <= {0.0, 1.0}
    chosen = np.take_along_axis(p, want, axis=1)
    w = chosen / (chosen if renormalize else p).sum(axis=1, keepdims=True)
    assert (np.abs(to64(weights) - w) <= 2.0 ** -22 * w).all()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("m,E,k,n", SHAPES)
@pytest.mark.parametrize("exponent", [66, 110, -80, -75])
def test_products_outside_fp32(m, E, k, n, exponent, renormalize):
    x, router = operands(m, E, n, exponent, m + E)
    logits = to64(x) @ to64(router).T
    nonzero = np.abs(logits[logits != 0])
    if exponent > 0:  # differences of 2^132 and more, finite in 64 bits
        assert nonzero.min() >= 2.0 ** (2 * exponent) and np.isfinite(logits).all()
        assert nonzero.max() > 2.0 ** 128
    else:             # below FP32's smallest steps
        assert nonzero.max() < 2.0 ** -100
        logits = logits * 2.0 ** (-2 * exponent)  # the same order; the weights are all alike
        ids, weights = dq4.dq4_moe_route(x.cuda(), router.cuda(), k, renormalize=renormalize)
        assert np.array_equal(ids.cpu().numpy(), np.argsort(-logits, axis=1, kind="stable")[:, :k])
        w = 1.0 / (k if renormalize else E)
        assert (np.abs(to64(weights) - w) <= 2.0 ** -22 * w).all()
        return
    checked(x, router, k, logits, renormalize)


@pytest.mark.parametrize("m", [2, 700])
def test_products_beyond_fp32_that_cancel(m):
    """2^140 - 2^140 + 1: finite logits, not infinities of both signs."""
    n, E = 24, 8
    x, r = np.zeros((m, n)), np.zeros((E, n))
    x[:, 3] = x[:, 11] = 2.0 ** 70
    x[:, 20] = 2.0 ** 60
    r[:, 3], r[:, 11] = 2.0 ** 70, -2.0 ** 70
    r[:, 20] = np.array([3, 7, 1, 7, 5, 2, 0, 4]) * 2.0 ** 48  # 2^108 apart: 32 bits below 2^140
    x, r = torch.from_numpy(x).bfloat16(), torch.from_numpy(r).bfloat16()
    checked(x, r, 3, to64(x) @ to64(r).T, True)
