"""C ABI of the LLM.int8 linear layer (include/dq4_int8.h), checked without a GPU:
every declared function is exported and bound, and bad arguments are rejected on
the host before anything is enqueued."""
import ctypes

import pytest

import block_wise_bit_amd as dq4
from libs import ensure_hip_library

P = ctypes.c_void_p
ONE = P(256)
BIG = 1 << 44


@pytest.fixture(scope="module")
def lib():
    return ensure_hip_library()


def test_exports_every_declared_function(lib):
    names = dq4.header_functions(dq4.INT8_HEADER_PATH)
    calls = {"dq4_int8_quant", "dq4_int8_linear", "dq4_int8_linear_backward"}
    assert set(names) == calls | {n + "_workspace_bytes" for n in calls}
    for name in names:
        assert hasattr(lib, name), name
        assert callable(getattr(dq4, name)), name


def test_quant_validation(lib):
    def call(x=ONE, m=4, k=64, ld=64, dtype=dq4.DQ4_F16, threshold=6.0, codes=ONE, ld_codes=64, scales=ONE,
             outliers=ONE, ws=ONE, ws_bytes=BIG):
        return lib.dq4_int8_quant(x, m, k, ld, dtype, threshold, codes, ld_codes, scales, outliers, ws, ws_bytes, None)
    assert call(m=0, threshold=0.0, outliers=None) == dq4.DQ4_OK
    for k in (dict(m=-1), dict(k=-1), dict(dtype=0), dict(dtype=3), dict(threshold=-1.0), dict(threshold=float("nan")),
              dict(outliers=None), dict(threshold=0.0), dict(x=None), dict(codes=None), dict(scales=None), dict(ld=63),
              dict(ld_codes=63), dict(ld=1 << 62), dict(ws_bytes=0), dict(ws=None), dict(ws=P(16))):
        assert call(**k) == dq4.DQ4_EINVAL, k
    for k in (dict(k=1 << 17, ld=1 << 17, ld_codes=1 << 17), dict(m=(1 << 21) + 1)):
        assert call(**k) == dq4.DQ4_EUNSUPPORTED, k


def test_linear_validation(lib):
    def call(codes=ONE, m=4, ld_codes=64, scales=ONE, CB=ONE, SCB=ONE, n=32, k=64, dtype=dq4.DQ4_BF16, x=None, ld_x=64,
             outliers=None, bias=None, residual=None, ld_r=32, y=ONE, ld_y=32, ws=ONE, ws_bytes=BIG):
        return lib.dq4_int8_linear(codes, m, ld_codes, scales, CB, SCB, n, k, dtype, x, ld_x, outliers, bias, residual,
                                   ld_r, y, ld_y, ws, ws_bytes, None)
    assert call(m=0) == dq4.DQ4_OK
    assert call(n=0) == dq4.DQ4_OK
    for k in (dict(m=-1), dict(n=-1), dict(k=-1), dict(dtype=0), dict(dtype=9), dict(codes=None), dict(scales=None),
              dict(CB=None), dict(SCB=None), dict(y=None), dict(x=ONE), dict(outliers=ONE), dict(ld_codes=63),
              dict(ld_y=31), dict(residual=ONE, ld_r=31), dict(x=ONE, outliers=ONE, ld_x=63), dict(ws=P(16)),
              dict(ws=None), dict(m=20, x=ONE, outliers=ONE, ws_bytes=0), dict(ws_bytes=-1), dict(ld_y=1 << 62)):
        assert call(**k) == dq4.DQ4_EINVAL, k
    for k in (dict(k=1 << 17, ld_codes=1 << 17), dict(n=(1 << 21) + 1, ld_y=1 << 22), dict(m=(1 << 21) + 1),
              dict(m=1 << 20, n=1 << 20, ld_y=1 << 20)):
        assert call(**k) == dq4.DQ4_EUNSUPPORTED, k


def test_backward_validation(lib):
    def call(CB=ONE, SCB=ONE, n=32, k=64, dtype=dq4.DQ4_F16, dy=ONE, m=4, ld_dy=32, dx=ONE, ld_dx=64, dbias=None,
             ws=ONE, ws_bytes=BIG):
        return lib.dq4_int8_linear_backward(CB, SCB, n, k, dtype, dy, m, ld_dy, dx, ld_dx, dbias, ws, ws_bytes, None)
    assert call(m=0) == dq4.DQ4_OK
    for k in (dict(m=-1), dict(n=-1), dict(k=-1), dict(dtype=0), dict(CB=None), dict(SCB=None), dict(dy=None),
              dict(dx=None), dict(ld_dy=31), dict(ld_dx=63), dict(ws_bytes=0), dict(ws=None), dict(ws=P(8))):
        assert call(**k) == dq4.DQ4_EINVAL, k
    for k in (dict(n=(1 << 21) + 1, ld_dy=1 << 22), dict(k=(1 << 21) + 1, ld_dx=1 << 22), dict(m=(1 << 21) + 1)):
        assert call(**k) == dq4.DQ4_EUNSUPPORTED, k


def test_workspace_sizes(lib):
    quant, linear = lib.dq4_int8_quant_workspace_bytes, lib.dq4_int8_linear_workspace_bytes
    assert quant(4, 1000, 0.0) == 0 and quant(1, 1000, 6.0) == 0 and quant(0, 1000, 6.0) == 0
    assert quant(2, 1000, 6.0) == 1024 and quant(2, 1 << 17, 6.0) == 0 and quant(2, 1000, float("nan")) == 0
    for bad in ((0, 64, 64), (4, 0, 64), (4, 64, -1), (1 << 22, 64, 64), (4, 1 << 22, 64), (4, 64, 1 << 17)):
        m, n, k = bad
        assert linear(ONE, m, 64, ONE, n, k, 1) == 0
    # a few tokens: the weight is read where it lies, whatever its alignment
    assert linear(ONE, 64, 4096, ONE, 4096, 4096, 0) == 0
    assert linear(P(1), 64, 4095, P(3), 4095, 4095, 0) == 0
    assert linear(P(1), 64, 8000, P(3), 4095, 8000, 0) == 0
    # outlier operands of 128 columns; up to 16 tokens are gathered in the product
    assert linear(ONE, 16, 4096, ONE, 4096, 4096, 1) == 0
    assert linear(ONE, 64, 4096, ONE, 4096, 4096, 1) == (4096 + 64) * 256
    # tiles: rows that are no multiple of 16 bytes take padded copies
    dense = linear(ONE, 2048, 4096, ONE, 4096, 4096, 0)
    assert linear(P(1), 2048, 4096, ONE, 4096, 4096, 0) == dense + 2048 * 4096
    assert linear(ONE, 2048, 4095, ONE, 4096, 4095, 0) == dense + (2048 + 4096) * 4096
    # rows that lie very far apart
    assert linear(ONE, 4, (1 << 22) + 16, ONE, 64, 64, 0) == 256
    back = lib.dq4_int8_linear_backward_workspace_bytes
    assert back(0, 64, 4, ONE, 64) == 0 and back(64, 64, 1 << 22, ONE, 64) == 0
    assert back(1000, 2048, 300, ONE, 1000) >= 1000 * 2048 * 2
    assert back(1000, 2048, 300, P(2), 1000) > back(1000, 2048, 300, ONE, 1000)


def test_binding_rejects_host_tensors(lib):
    torch = pytest.importorskip("torch")
    x, i8, f = torch.zeros((4, 16), dtype=torch.float16), torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        dq4.dq4_int8_quant(x)
    with pytest.raises(ValueError):
        dq4.dq4_int8_linear(i8, f, i8, f)
    with pytest.raises(ValueError):
        dq4.dq4_int8_linear_backward(x[:, :4], i8, f)
