"""The workspace of dq4_int8_linear against the outlier operands that its kernels
read (no GPU).

With more than 16 tokens the operands of the first 128 outlier columns are
gathered into the workspace: four chunks of 1 KiB for each 16 rows of the weight,
then for each tile of 16 tokens.  The row kernels (up to 64 tokens) work on 1, 2 or
4 tiles of tokens at a time and read the operands of all of them, whether or not
the last ones hold a token, so the workspace has to hold all of them.
"""
import ctypes

import pytest

from libs import ensure_hip_library

P = ctypes.c_void_p
CHUNKS = 4          # of 32 outlier columns
FRAGMENT = 1024     # bytes of a chunk of 16 rows
SHAPES = [(64, 192, 256, 256), (100, 64, 256, 256), (129, 1024, 256, 256), (8777, 4096, 256, 256), (49104, 4096, 256, 256),
          (300, 100, 256, 256), (47, 1377, 1, 3), (64, 8000, 1, 256)]  # n_out, n_in, addresses of codes and CB


@pytest.fixture(scope="module")
def lib():
    return ensure_hip_library()


def ceil_div(a, b):
    return -(-a // b)


def row_kernel_tiles(m):
    return 1 if m <= 16 else 2 if m <= 32 else 4


def last_read(m, n, tiles, base):
    """Behind the last byte of the token operands that a row kernel reads, their
    region starting at `base` of the workspace."""
    return max(base + ((t * CHUNKS + c) * 64 + lane) * 16 + 16
               for t in range(tiles) for c in range(CHUNKS) for lane in (0, 63))


def overruns(m, n, held):
    base = ceil_div(n, 16) * CHUNKS * FRAGMENT
    return last_read(m, n, row_kernel_tiles(m), base) > held


@pytest.mark.parametrize("n,k,codes_at,CB_at", SHAPES)
def test_row_kernels_read_inside_the_workspace(lib, n, k, codes_at, CB_at):
    for m in range(17, 65):
        if m > 32 and k > 4096 and codes_at % 16 == 0 and CB_at % 16 == 0 and k % 16 == 0:
            continue  # tiles
        held = lib.dq4_int8_linear_workspace_bytes(P(codes_at), m, k, P(CB_at), n, k, 1)
        assert held % (CHUNKS * FRAGMENT) == 0
        assert not overruns(m, n, held), (m, n, k, held)
        # and nothing but the operands
        assert held == (ceil_div(n, 16) + row_kernel_tiles(m)) * CHUNKS * FRAGMENT, (m, n, k)


def test_tiles_of_many_tokens_read_inside_the_workspace(lib):
    """Tiles of 64, 128 or 256 tokens leave out the 16 tokens at a time that lie
    behind the last one: the operands of ceil(m / 16) are read."""
    for m in (65, 66, 80, 81, 100, 128, 129, 150, 300, 1030):
        for n, k in ((129, 1024), (1000, 4096), (256, 64)):
            plain = lib.dq4_int8_linear_workspace_bytes(P(256), m, k, P(256), n, k, 0)
            held = lib.dq4_int8_linear_workspace_bytes(P(256), m, k, P(256), n, k, 1)
            assert held - plain == (ceil_div(n, 128) * 8 + ceil_div(m, 16)) * CHUNKS * FRAGMENT, (m, n, k)


def test_planted_size_for_tiles_with_tokens_is_found():
    for m in range(17, 65):
        held = (ceil_div(49104, 16) + ceil_div(m, 16)) * CHUNKS * FRAGMENT
        assert overruns(m, 49104, held) == (33 <= m <= 48)
