"""Index arithmetic of the 128-row tile kernel (tile_rows_kernel in
block_wise_bit_amd/csrc/dq4_linear_fused.hip), restated on the CPU (no GPU).

A workgroup walks the chunks of 512 k of its part of the summed index.  While
it multiplies a chunk it loads the next one (at the end: the same one again)
and looks up that chunk's first steps, through a table in LDS of 256 entries
of 256 bytes and a row of 256 zero bytes behind them; x's fragments of four
steps at a time go to one of two stages in LDS.  These checks pin that every
lookup stays inside the table, that a stage is never written while it is read
and holds what its reader expects, and that the parts of a split tile lie apart
in the workspace and are summed from where they were written.  A planted
mistake of each kind is found.
"""
from __future__ import annotations

import itertools

import pytest

SPAN = 512
TABLE = 256 * 32 * 8      # 256 entries of 32 copies of a pair of floats
ZEROS = 256               # the row of zeros behind it

# (n_in, splits): whole chunks, a last chunk that ends in every quarter and
# piece, parts of unequal length, parts of one chunk
WALKS = [(512, 1), (1024, 2), (32, 1), (544, 1), (544, 2), (640, 1), (2048, 4), (4128, 1), (4128, 3), (4128, 9),
         (6176, 5), (8192, 1), (66560, 16), (160, 1), (384 + 512 * 6, 7)]


def parts(n_in, splits):
    chunks = -(-n_in // SPAN)
    assert splits <= chunks
    for s in range(splits):
        yield s * chunks // splits, (s + 1) * chunks // splits


def table_reads(n_in, begin, end, look, next_chunk):
    """(address span of a lookup) over the walk: 256 bytes per code byte, a
    lane's copy within them.  A piece of 32 k beyond the row was loaded as
    zeros; any other may hold any byte."""
    def beyond(chunk, g, piece):
        return chunk * SPAN + 128 * g + 32 * piece >= n_in

    def read(held, told, g, step):
        base = TABLE if beyond(told, g, step // 4) else 0
        top = 0 if beyond(held, g, step // 4) else 255
        for lane_byte in (0, 31 * 8):           # the first and last copy; 8 bytes are read
            yield base + lane_byte, base + 256 * top + lane_byte + 8
    for g in range(4):
        for i in range(look):
            yield from read(begin, begin, g, i)
        for c in range(begin, end):
            held = c + 1 if c + 1 < end else c
            for st in range(16):
                if st + look < 16:
                    yield from read(c, c, g, st + look)
                else:
                    yield from read(held, next_chunk(c, end), g, st + look - 16)


def outside(n_in, splits, look, next_chunk):
    return [(a, b) for begin, end in parts(n_in, splits)
            for a, b in table_reads(n_in, begin, end, look, next_chunk) if a < 0 or b > TABLE + ZEROS]


@pytest.mark.parametrize("look", [1, 2])
@pytest.mark.parametrize("n_in,splits", WALKS)
def test_lookups_stay_inside_the_table(n_in, splits, look):
    assert not outside(n_in, splits, look, lambda c, end: c + 1 if c + 1 < end else c)


def test_planted_chunk_past_the_end_is_found():
    """Told the chunk after the last while the registers hold the last again,
    the lookup takes nonzero codes for a piece beyond the row."""
    assert any(outside(n_in, splits, 1, lambda c, end: c + 1) for n_in, splits in WALKS)


def stage_walk(begin, end, after_last):
    """For each quarter q of a chunk: (stage read, quarter it must hold, stage
    written meanwhile, quarter written)."""
    held = {(4 * begin) & 1: 4 * begin}
    for c in range(begin, end):
        for j in range(4):
            q = 4 * c + j
            to = q + 1 if q + 1 < 4 * end else after_last(q)
            assert held[q & 1] == q
            yield q & 1, to & 1
            held[to & 1] = to


@pytest.mark.parametrize("n_in,splits", WALKS)
def test_stages_are_not_written_while_read(n_in, splits):
    for begin, end in parts(n_in, splits):
        assert begin < end
        assert all(read != written for read, written in stage_walk(begin, end, lambda q: q - 1))
        # the kernel's last load reads x's fragments of its own chunk: in range
        chunks = -(-n_in // SPAN)
        assert 0 <= 4 * begin and 4 * end - 2 < 4 * chunks


def test_planted_stage_is_found():
    assert any(read == written for read, written in stage_walk(0, 2, lambda q: q))


@pytest.mark.parametrize("rest,splits", [(1, 2), (3, 16), (128, 2), (37, 5)])
def test_split_sums_lie_apart_and_are_found_again(rest, splits):
    """Units of 1 KiB (64 lanes of four floats)."""
    def written(split, at, wave, t, f):
        return ((split * rest + at) * 8 + wave) * 16 + t * 2 + f

    def summed(split, at, wave, t, f):
        return ((at * 8 + wave) * 8 + t) * 2 + split * (rest * 8 * 8 * 2) + f
    seen = set()
    for split, at, wave, t, f in itertools.product(range(splits), range(rest), range(8), range(8), range(2)):
        u = written(split, at, wave, t, f)
        assert u == summed(split, at, wave, t, f)
        seen.add(u)
    assert len(seen) == splits * rest * 128 and max(seen) * 1024 < splits * rest * 128 * 256 * 4
