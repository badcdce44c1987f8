"""C ABI of the mixture-of-experts layer (include/dq4_moe.h), checked without a
GPU: every declared function is exported and bound, and bad arguments are rejected
on the host before anything is enqueued."""
import ctypes

import pytest

import block_wise_bit_amd as dq4
from libs import ensure_hip_library
from test_linear_abi import weight

P = ctypes.c_void_p
ONE = P(256)
BIG = 1 << 44


@pytest.fixture(scope="module")
def lib():
    return ensure_hip_library()


def test_exports_every_declared_function(lib):
    names = dq4.header_functions(dq4.MOE_HEADER_PATH)
    assert set(names) == {"dq4_moe_route", "dq4_moe_fused", "dq4_moe_route_workspace_bytes",
                          "dq4_moe_fused_workspace_bytes"}
    for name in names:
        assert hasattr(lib, name), name
        assert callable(getattr(dq4, name)), name


def test_route_validation(lib):
    def call(x=ONE, m=4, n=64, ld=64, dtype=dq4.DQ4_F16, router=ONE, bias=None, E=8, k=2, ids=ONE, weights=ONE,
             ws=ONE, ws_bytes=BIG):
        return lib.dq4_moe_route(x, m, n, ld, dtype, router, bias, E, k, 1, ids, weights, ws, ws_bytes, None)
    assert call(m=0) == dq4.DQ4_OK
    for k in (dict(m=-1), dict(n=-1), dict(E=-1), dict(E=0), dict(k=0), dict(k=9), dict(dtype=0), dict(dtype=3),
              dict(x=None), dict(router=None), dict(ids=None), dict(weights=None), dict(ld=63), dict(ld=1 << 62), dict(ws=None),
              dict(ws=P(16)), dict(ws_bytes=255)):
        assert call(**k) == dq4.DQ4_EINVAL, k
    for k in (dict(E=513), dict(E=20, k=17), dict(m=(1 << 21) + 1), dict(n=(1 << 17) + 1, ld=1 << 18)):
        assert call(**k) == dq4.DQ4_EUNSUPPORTED, k


def test_experts_validation(lib):
    def call(g=None, u=None, d=None, E=4, n_ff=32, n_in=64, dtype=dq4.DQ4_BF16, act=dq4.DQ4_ACT_SILU, x=ONE, m=4,
             ld_x=64, ids=ONE, weights=ONE, k=2, residual=None, ld_r=64, y=ONE, ld_y=64, ws=ONE, ws_bytes=BIG,
             null=False):
        at = lambda w: None if null else ctypes.byref(w or weight())  # noqa: E731
        return lib.dq4_moe_fused(at(g), at(u), at(d), E, n_ff, n_in, dtype, act, x, m, ld_x, ids, weights, k, residual,
                                 ld_r, y, ld_y, ws, ws_bytes, None)
    assert call(m=0) == dq4.DQ4_OK
    assert call(n_in=0) == dq4.DQ4_OK
    for k in (dict(null=True), dict(m=-1), dict(n_ff=-1), dict(n_in=-1), dict(E=0), dict(k=0), dict(dtype=0),
              dict(act=0), dict(act=5), dict(x=None), dict(y=None), dict(ids=None), dict(weights=None), dict(ld_x=63),
              dict(ld_y=63), dict(residual=ONE, ld_r=63), dict(g=weight(packed=None)), dict(u=weight(ptr=None)),
              dict(d=weight(codebook4=None)), dict(n_ff=0, d=weight(scale_codebook=None)), dict(ws_bytes=0), dict(ws=None),
              dict(ws=P(16))):
        assert call(**k) == dq4.DQ4_EINVAL, k
    for k in (dict(E=513), dict(k=17), dict(m=65), dict(n_ff=(1 << 17) + 1), dict(n_in=(1 << 17) + 1, ld_x=1 << 18, ld_y=1 << 18),
              dict(E=512, n_ff=1 << 17, n_in=1 << 17, ld_x=1 << 17, ld_y=1 << 17), dict(g=weight(blocksize=128)),
              dict(d=weight(blocksize=48)), dict(u=weight(nested=128))):
        assert call(**k) == dq4.DQ4_EUNSUPPORTED, k


def test_workspace_sizes(lib):
    f = lib.dq4_moe_fused_workspace_bytes
    for bad in ((0, 32, 64, 4, 2), (4, -1, 64, 4, 2), (4, 32, 0, 4, 2), (4, 32, 64, 0, 2), (4, 32, 64, 4, 0),
                (513, 32, 64, 4, 2), (4, 32, 64, 65, 2), (4, 32, 64, 4, 17)):
        assert f(*bad) == 0, bad
    # a tile of x (512 k a chunk, 16 KiB) and one of h for each expert
    assert f(64, 1024, 2048, 1, 8) == 256 + 256 + 512 + 512 + 8 * 4 * 16384 + 8 * 2 * 16384
    # 64 tokens: a tile per expert and one more for every 16 choices
    assert f(8, 512, 512, 64, 2) == 256 + 256 + 2 * 1024 + 16 * 16384 + 16 * 16384
    assert f(512, 1 << 10, 1 << 10, 64, 16) > 0
    g = lib.dq4_moe_route_workspace_bytes
    assert g(1, 8) == 256 and g(100, 64) == 51200 and g(0, 8) == 0 and g(4, 513) == 0 and g((1 << 21) + 1, 8) == 0


def test_binding_rejects_host_tensors(lib):
    torch = pytest.importorskip("torch")
    u8, f = torch.zeros(4096, dtype=torch.uint8), torch.zeros(256)
    w = dict(packed=u8, scale_codes=u8, nested_absmax=f, scale_codebook=f, codebook4=f[:16], offset=0.0)
    x = torch.zeros((2, 32), dtype=torch.float16)
    with pytest.raises(ValueError):
        dq4.dq4_moe_route(x, x, 1)
    with pytest.raises(ValueError):
        dq4.dq4_moe_fused(w, w, w, 2, 32, 32, 64, x, torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1)))
