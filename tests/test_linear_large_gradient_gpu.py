"""The bias gradient of a matrix of more than 2^34 elements in odd rows (32
GiB): one thread a column and eight rows would be 2^32 threads, more than one
launch can hold."""
from __future__ import annotations

import pytest

import block_wise_bit_amd as dq4
from block_wise_bit_amd import inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


def test_sums_of_more_threads_than_a_launch_holds():
    m, n = 1 << 20, 16385
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("not enough free memory")
    x = inputs.make_inputs(n * 64, 64, "nf4", 0.03, seed=5, n_rows=n, n_cols=64)
    w = dict(dq4.to_device(x), offset=float(x.offset))
    print(f"dbias of {m} x {n}", flush=True)
    dy = torch.ones((m, n), dtype=torch.bfloat16, device="cuda")
    # rows and columns that only the last workgroups reach
    dy[m - 1, n - 1], dy[m - 33, 7], dy[12345, n - 2] = 3.0, -2.0, 5.0
    dx, dz, db = dq4.dq4_linear_fused_backward(**w, n_out=n, n_in=0, blocksize=64, dy=dy, bias_grad=True)
    assert dx.shape == (m, 0) and dz is dy
    want = torch.full((n,), float(m), device="cuda")    # sums of small whole numbers: exact
    want[n - 1] += 2.0
    want[7] -= 3.0
    want[n - 2] += 4.0
    assert torch.equal(db, want)
    del dy, dz
    torch.cuda.empty_cache()
