"""Calls that would take 2^32 threads or more, of which a launch runs only a
part, without an error."""
from __future__ import annotations

import pytest

import block_wise_bit_amd as dq4

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


def test_out_prod_of_more_workgroups_than_a_launch_holds():
    """2^31 + 128 columns, a workgroup each 128: refused, nothing written."""
    n_rows, n_cols, bs = 2, (1 << 31) + 128, 4096
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    n = n_rows * n_cols
    print(f"out_prod {n_rows} x {n_cols}", flush=True)
    w = dict(packed=torch.full((n // 2,), 0x52, dtype=torch.uint8, device="cuda"),
             scale_codes=torch.full((-(-n // bs),), 3, dtype=torch.uint8, device="cuda"),
             nested_absmax=torch.ones(-(-n // bs // 256) + 1, device="cuda"),
             scale_codebook=torch.full((256,), 2.0, device="cuda"),
             codebook4=torch.arange(16, dtype=torch.float32, device="cuda"), offset=1.0)
    src1 = torch.ones((n_rows, 1), device="cuda")
    dst = torch.full((1, n_cols), 7.0, device="cuda")
    with pytest.raises(ValueError):
        dq4.dq4_out_prod_fused(**w, n_rows=n_rows, n_cols=n_cols, blocksize=bs, src1=src1, dst=dst)
    torch.cuda.synchronize()
    assert bool((dst == 7.0).all())
    # one tile fewer than the most: codes 2 and 5 times a scale of 3, two rows
    cols = ((1 << 24) - 1) * 128
    dq4.dq4_out_prod_fused(**w, n_rows=n_rows, n_cols=cols, blocksize=bs, src1=src1, dst=dst.view(-1)[:cols].view(1, cols))
    got = dst.view(-1)[:cols].view(-1, 2)
    assert bool((got[:, 0] == 12.0).all()) and bool((got[:, 1] == 30.0).all())
    del w, dst, got, src1
    torch.cuda.empty_cache()
