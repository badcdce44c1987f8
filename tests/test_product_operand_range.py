"""The products' left operand as a buffer (fragment_product_kernel and
fragment_product_wide_kernel in block_wise_bit_amd/csrc/dq4_linear_fused.hip),
restated on the CPU, and rows without columns on the GPU.

A workgroup reads 256 rows at most through a buffer of ((rows - 1) ld + k) 2
bytes, with 32-bit offsets; rows and k beyond the matrix get the offset 2^31,
which has to lie past the buffer.
"""
from __future__ import annotations

import numpy as np
import pytest

import block_wise_bit_amd as dq4
from block_wise_bit_amd import inputs

NOTHING = 0x80000000
MAX_LD = 1 << 22


def product_ld(ld, m, k):
    return ld if m > 1 and k > 0 else k


def buffer_bytes(rows, ld, k):
    return (((rows - 1) * ld + k) * 2) & 0xFFFFFFFF


CASES = [(m, ld, k) for m in (1, 2, 17, 256, 1 << 21) for k in (0, 8, 1000, 1 << 21)
         for ld in (k, 1 << 21, MAX_LD, 1 << 23, 1 << 40, 1 << 61) if ld >= k]


def read_in_place(m, ld, k):
    """No copy is made of it (aligned rows of whole 16-byte pieces)."""
    return not (m > 1 and ld > MAX_LD and k > 0)


@pytest.mark.parametrize("m,ld,k", [c for c in CASES if read_in_place(*c)])
def test_what_is_not_there_lies_past_the_buffer(m, ld, k):
    rows = min(m, 256)
    ld = product_ld(ld, m, k)
    size = ((rows - 1) * ld + k) * 2
    assert size == buffer_bytes(rows, ld, k) <= NOTHING
    if k:
        assert ((rows - 1) * ld + k - 8) * 2 + 16 <= size       # the last 16 bytes of the last row


def test_planted_stride_without_columns_is_found():
    """The stride of rows without columns taken as given: the buffer covers 2^31."""
    assert any(buffer_bytes(min(m, 256), ld, k) > NOTHING for m, ld, k in CASES if k == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("ld", [1, 1 << 22, 1 << 23, 1 << 40])
@pytest.mark.parametrize("m", [2, 70, 300])
def test_rows_without_columns_on_the_gpu(m, ld):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()
    print(f"rows without columns m={m} ld={ld}", flush=True)
    x = inputs.make_inputs(520 * 128, 64, "nf4", 0.03, seed=3, n_rows=520, n_cols=128)
    w = dict(dq4.to_device(x), offset=float(x.offset))
    none = torch.as_strided(torch.zeros(8, dtype=torch.float16, device="cuda"), (m, 0), (ld, 1))
    bias = torch.from_numpy(np.arange(520, dtype=np.float16)).cuda()
    y = dq4.dq4_linear_fused(**w, n_out=520, n_in=0, blocksize=64, x=none, bias=bias)
    assert torch.equal(y, bias.expand(m, 520))
    assert bool((dq4.dq4_gated_fused(w, w, 520, 0, 64, none) == 0).all())
    dx, _, db = dq4.dq4_linear_fused_backward(**w, n_out=0, n_in=128, blocksize=64, dy=none, bias_grad=True)
    assert dx.shape == (m, 128) and bool((dx == 0).all()) and db.numel() == 0
    dx, _, _ = dq4.dq4_gated_fused_backward(w, w, 0, 128, 64, none, none, none)
    assert dx.shape == (m, 128) and bool((dx == 0).all())
