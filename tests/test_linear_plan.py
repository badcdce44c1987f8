"""The restated choice of kernels (linear_plan.py) against the library's
workspace sizes, and what the shapes of the route tests cover.  No GPU."""
import ctypes
import random

import pytest

import block_wise_bit_amd as dq4
import linear_plan as plan
from libs import ensure_hip_library

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return ensure_hip_library()


def shapes():
    rng = random.Random(11)
    for m, n, k, _ in plan.TILE_LINEAR + plan.TILE_GATED:
        yield m, n, k
    for m, n, k in plan.PRODUCTS + plan.PRODUCTS_GATED + plan.PRODUCTS_GATED_BACKWARD:
        yield m, n, k
        yield m, k, n
    for _ in range(400):
        def size(most):
            return max(1, int(round(most ** rng.random())))
        step = rng.choice([1, 8, 32, 64])
        yield size(4096), max(step, size(40000) // step * step), max(step, size(40000) // step * step)


def test_workspace_sizes_follow_the_restated_plan(lib):
    w = dq4.Dq4Weight(16, 16, 16, 16, 16, 0.03, 64, 256)
    r = ctypes.byref(w)
    for m, n, k in shapes():
        for least in (0, 1):
            for at in (256, 2):
                ok = at == 256
                got = lib.dq4_linear_fused_workspace_bytes(r, n, k, m, P(at), k, least)
                assert got == plan.forward_workspace(m, n, k, False, least, ok), (m, n, k, least, at)
                got = lib.dq4_gated_fused_workspace_bytes(r, r, n, k, m, P(at), k, least)
                assert got == plan.forward_workspace(m, n, k, True, least, ok), (m, n, k, least, at)
                got = lib.dq4_linear_fused_backward_workspace_bytes(r, n, k, m, P(at), n, least)
                assert got == plan.backward_workspace(m, n, k, False, least, ok), (m, n, k, least, at)
                got = lib.dq4_gated_fused_backward_workspace_bytes(r, r, n, k, m, P(at), P(at), n, least)
                assert got == plan.backward_workspace(m, n, k, True, least, ok), (m, n, k, least, at)


@pytest.mark.parametrize("shapes,gated", [(plan.TILE_LINEAR, False), (plan.TILE_GATED, True)])
def test_tile_shapes_cover_every_cut(shapes, gated):
    kinds = {plan.tile_kind(*s, gated) for s in shapes}
    assert kinds == {(cut, s) for cut in ("whole", "whole, several", "both", "split") for s in (2, 4)}


@pytest.mark.parametrize("shapes,group,weights", [(plan.PRODUCTS, 128, 1), (plan.PRODUCTS_GATED, 64, 1),
                                                  (plan.PRODUCTS_GATED_BACKWARD, 128, 2)])
def test_product_shapes_cover_every_tile(shapes, group, weights):
    seen = set()
    for m, n, k in shapes:
        tile, splits, _ = plan.product_plan(m, plan.ceil_div(n, group), weights * plan.ceil_div(k, 64))
        seen.add((tile, splits > 1))
    assert seen == {(t, s) for t in range(3) for s in (False, True)}
