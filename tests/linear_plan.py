"""How the fused linear and gated calls choose their kernels, restated
(route_of, tile_plan, plan_of and column_plan in
block_wise_bit_amd/csrc/dq4_linear_fused.hip), so that a test can say which
kernel its shape is meant for.  test_linear_plan.py holds this against the
library's workspace sizes; 256 compute units, 4-byte aligned codes.
"""
from __future__ import annotations

CUS = 256


def ceil_div(a, b):
    return -(-a // b)


TILE_COLS, TILE_ROWS, RESIDENT, CHUNK_US = (256, 128, 128), (256, 128, 64), (1, 2, 3), (1.78, 1.40, 1.80)


def product_plan(m, groups, chunks):
    """(tile, splits, cost) of the product over decoded fragments."""
    best = (2, 1, 1e300)
    for tile in range(3):
        tiles = ceil_div(groups * 128, TILE_COLS[tile]) * ceil_div(m, TILE_ROWS[tile])
        for splits in range(1, 17):
            if splits > 1 and splits * 2 > chunks:
                break
            rounds = ceil_div(tiles * splits, CUS * RESIDENT[tile])
            cost = rounds * (ceil_div(chunks, splits) * CHUNK_US[tile] + 2.0)
            if splits > 1:
                cost += 3.0 + splits * m * (groups * 128) * 8.0 / 4e6
            if cost < best[2]:
                best = (tile, splits, cost)
    return best


def tile_plan(m, n_out, n_in, gated):
    """(whole tiles, split tiles, splits, cost) of the 128-row tiles."""
    tiles, chunks = ceil_div(n_out, 128 if gated else 256) * ceil_div(m, 128), ceil_div(n_in, 512)
    whole = tiles // CUS * CUS
    rest = tiles - whole
    best = (tiles, 0, 1, 1e300)
    for splits in range(1, min(16, chunks) + 1):
        cost = (whole // CUS) * (chunks * 8.0 + 9.0) + ceil_div(rest * splits, CUS) * (ceil_div(chunks, splits) * 8.0 + 9.0)
        if splits > 1:
            cost += 3.0 + rest * splits * (128 * 256 * 8.0 / 4e6)
        if cost < best[3]:
            best = (tiles, 0, 1, cost) if splits == 1 else (whole, rest, splits, cost)
    return best


def forward_groups(n_out, gated):
    return ceil_div(n_out, 64 if gated else 128)


def forward_route(m, n_out, n_in, gated):
    if m > 1024 or n_in == 0 or n_in % 8:
        return "product"
    if n_in % 32:
        return "ragged" if m <= 64 else "product"
    if m <= 2 and n_in <= 32768:
        return "token"
    if m <= 64:
        return "batch"
    decode = 5.0 + n_out * n_in * (2 if gated else 1) * 4.8e-7
    product = product_plan(m, forward_groups(n_out, gated), ceil_div(n_in, 64))[2] + decode
    return "tile" if tile_plan(m, n_out, n_in, gated)[3] < product else "product"


def backward_route(m, n_out, n_in):
    return "columns" if m <= 128 and n_out > 0 and n_in > 0 and n_in % 8 == 0 else "product"


def x_fragment_bytes(m, k):
    tf = 1 if m <= 16 else 2 if m <= 32 else 4 if m <= 64 else 8
    return ceil_div(m, 16 * tf) * ceil_div(k, 512) * 16 * tf * 1024


def window_bytes(m, groups, all_groups, chunks):
    tile, splits, _ = product_plan(m, all_groups, chunks)
    size = groups * chunks * 16384
    if splits > 1:
        size += splits * ceil_div(groups * 128, TILE_COLS[tile]) * TILE_COLS[tile] * ceil_div(m, TILE_ROWS[tile]) * TILE_ROWS[tile] * 4
    return size


def aligned(n, to=256):
    return ceil_div(n, to) * to


def padded_copy_bytes(m, k):
    return aligned(m * ceil_div(k, 64) * 64 * 2)


def forward_workspace(m, n_out, n_in, gated, least, x_aligned):
    route = forward_route(m, n_out, n_in, gated)
    copy = 0 if x_aligned and n_in % 8 == 0 else padded_copy_bytes(m, n_in)
    if route == "product":
        groups = forward_groups(n_out, gated)
        return copy + window_bytes(m, min(groups, 2) if least else groups, groups, ceil_div(n_in, 64))
    if route in ("token", "ragged"):
        return copy
    whole, rest, splits, _ = tile_plan(m, n_out, n_in, gated)
    sums = splits * rest * 128 * 256 * 4 if route == "tile" and splits > 1 else 0
    return x_fragment_bytes(m, n_in) + sums


def backward_workspace(m, n_out, n_in, gated, least, dz_aligned):
    weights = 2 if gated else 1
    bias = 0 if gated else aligned(ceil_div(m, 32) * n_out * 4)
    if backward_route(m, n_out, n_in) == "columns":
        tf = 1 if m <= 16 else 2
        slices, steps, groups = ceil_div(m, 16 * tf), ceil_div(n_out, 32), ceil_div(n_in, 128)
        splits = max(1, min(CUS // (groups * slices), ceil_div(steps * weights, 8)))
        return bias + weights * slices * steps * tf * 1024 + splits * groups * slices * 8 * tf * 1024
    copy = 0 if dz_aligned and n_out % 8 == 0 else weights * padded_copy_bytes(m, n_out)
    groups = ceil_div(n_in, 128)
    return bias + copy + window_bytes(m, min(groups, 2) if least else groups, groups, weights * ceil_div(n_out, 64))


# ----------------------------------------------------------------------------
# shapes of the tests that are meant for one kernel
# ----------------------------------------------------------------------------
# (m, n_out, n_in, blocksize): the 128-row tiles, whole and split along k in
# every way, one and more to a workgroup, blocks looked up per 64 k (S = 2) and
# per 32 k (S = 4), rows, weight rows and chunks that end inside a tile
TILE_LINEAR = [
    (65, 28672, 544, 64),      # whole, S = 4, a last chunk of one piece
    (130, 16400, 2048, 64),    # whole, S = 2
    (257, 33000, 1056, 32),    # whole, more tiles than workgroups, S = 4
    (257, 33000, 2048, 4096),  # the same, S = 2
    (385, 16400, 2048, 128),   # a round of whole tiles and one of split ones, S = 2
    (129, 33000, 1056, 64),    # the same, S = 4
    (100, 300, 6176, 32),      # split alone, uneven parts, S = 4
    (65, 100, 8192, 256),      # split alone, one chunk a part, S = 2
]
TILE_GATED = [
    (65, 16400, 544, 64), (129, 8200, 2048, 64), (257, 16400, 1056, 32), (257, 16400, 2048, 4096),
    (129, 16400, 2048, 128), (129, 16400, 1056, 64), (65, 300, 6176, 32), (129, 100, 8192, 256),
]


def tile_kind(m, n_out, n_in, blocksize, gated):
    """(how the tiles are cut, S) of a shape that takes the 128-row tiles."""
    assert forward_route(m, n_out, n_in, gated) == "tile", (m, n_out, n_in, gated)
    whole, rest, splits, _ = tile_plan(m, n_out, n_in, gated)
    cut = ("split" if whole == 0 else "both") if splits > 1 else "whole" if whole <= CUS else "whole, several"
    return cut, 2 if blocksize >= 64 and n_in % 64 == 0 else 4


# (m, output columns, summed index), odd widths: every tile of the product over
# decoded fragments, one part and several
PRODUCTS = [(130, 33001, 65), (130, 12801, 2049), (5, 65, 33), (3, 127, 1001), (5, 70001, 65), (2, 9001, 1377)]
PRODUCTS_GATED = [(130, 16501, 65), (130, 8201, 1377), (5, 65, 33), (3, 127, 515), (2, 33001, 65), (2, 4097, 1377)]
PRODUCTS_GATED_BACKWARD = [(130, 33001, 33), (130, 8201, 1377), (5, 65, 33), (3, 127, 515), (5, 70001, 33), (2, 9001, 515)]
