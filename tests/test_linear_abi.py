"""C ABI of the fused linear and gated calls (include/dq4_linear.h), checked
without a GPU: every declared function is exported and bound, and bad
arguments are rejected on the host before anything is enqueued."""
import ctypes

import pytest

import block_wise_bit_amd as dq4
from libs import ensure_hip_library

P = ctypes.c_void_p
ONE = P(256)


@pytest.fixture(scope="module")
def lib():
    return ensure_hip_library()


def test_exports_every_declared_function(lib):
    names = dq4.header_functions(dq4.LINEAR_HEADER_PATH)
    calls = {"dq4_linear_fused", "dq4_linear_fused_backward", "dq4_gated_fused",
             "dq4_gated_fused_backward"}
    assert set(names) == calls | {n + "_workspace_bytes" for n in calls}
    for name in names:
        assert hasattr(lib, name), name
        assert callable(getattr(dq4, name)), name


def weight(ptr=16, blocksize=64, nested=256, **missing):
    fields = dict.fromkeys(("packed", "scale_codes", "nested_absmax", "scale_codebook", "codebook4"), ptr)
    fields.update(missing)
    return dq4.Dq4Weight(*fields.values(), 0.03, blocksize, nested)


BIG = 1 << 40   # more workspace than any of these calls asks for


def linear(lib, n_out=64, n_in=128, dtype=dq4.DQ4_F16, act=0, x=ONE, m=4, ld_x=128, bias=None, res=None,
           ld_res=64, y=ONE, ld_y=64, pre=None, ld_pre=64, ws=ONE, ws_bytes=0, w=None, null_w=False):
    w = None if null_w else ctypes.byref(w or weight())
    return lib.dq4_linear_fused(w, n_out, n_in, dtype, act, x, m, ld_x, bias, res, ld_res, y, ld_y,
                                pre, ld_pre, ws, ws_bytes, None)


def test_linear_validation(lib):
    def call(**k):
        return linear(lib, **k)
    assert call(m=0) == dq4.DQ4_OK
    assert call(n_out=0) == dq4.DQ4_OK
    assert call(m=300) == dq4.DQ4_EINVAL                          # no workspace
    assert call(ws=None, ws_bytes=BIG) == dq4.DQ4_EINVAL
    assert call(ws=P(16), ws_bytes=BIG) == dq4.DQ4_EINVAL         # not 256-byte aligned
    for k in (dict(null_w=True), dict(x=None), dict(y=None), dict(m=-1), dict(n_out=-1), dict(n_in=-1),
              dict(dtype=dq4.DQ4_F32), dict(dtype=7), dict(act=5), dict(act=-1), dict(ld_x=127),
              dict(ld_y=63), dict(res=ONE, ld_res=63), dict(pre=ONE, ld_pre=63), dict(w=weight(ptr=None)),
              dict(w=weight(scale_codes=None)), dict(w=weight(codebook4=None)), dict(ld_x=1 << 62)):
        assert call(**dict(dict(ws_bytes=BIG), **k)) == dq4.DQ4_EINVAL, k
    for k in (dict(w=weight(blocksize=48)), dict(w=weight(blocksize=16)), dict(w=weight(nested=128)),
              dict(n_out=(1 << 21) + 1), dict(n_in=(1 << 21) + 1), dict(m=(1 << 21) + 1),
              dict(m=1 << 19, n_out=1 << 21)):
        assert call(**dict(dict(ws_bytes=BIG), **k)) == dq4.DQ4_EUNSUPPORTED, k


def test_linear_backward_validation(lib):
    def call(n_out=64, n_in=128, dtype=dq4.DQ4_BF16, act=dq4.DQ4_ACT_GELU, dy=ONE, m=4, ld_dy=64, pre=ONE,
             ld_pre=64, dx=ONE, ld_dx=128, dz=ONE, ld_dz=64, dbias=None, ws=ONE, ws_bytes=BIG, w=None):
        return lib.dq4_linear_fused_backward(ctypes.byref(w or weight()), n_out, n_in, dtype, act, dy, m,
                                             ld_dy, pre, ld_pre, dx, ld_dx, dz, ld_dz, dbias, ws, ws_bytes,
                                             None)
    assert call(m=0) == dq4.DQ4_OK
    for k in (dict(ws_bytes=0), dict(ws=None), dict(dy=None), dict(pre=None), dict(dz=None), dict(dx=None),
              dict(act=0), dict(act=9), dict(ld_dy=63), dict(ld_pre=63), dict(ld_dz=63), dict(ld_dx=127),
              dict(m=-1), dict(dtype=0), dict(w=weight(packed=None))):
        assert call(**k) == dq4.DQ4_EINVAL, k          # act=0: dz is dy, none may be given
    assert call(w=weight(blocksize=33)) == dq4.DQ4_EUNSUPPORTED


def test_gated_validation(lib):
    def call(gate=None, up=None, n_ff=64, n_in=128, dtype=dq4.DQ4_F16, act=dq4.DQ4_ACT_SILU, x=ONE, m=4,
             ld_x=128, h=ONE, ld_h=64, g=None, u=None, ld_pre=64, ws=ONE, ws_bytes=BIG):
        return lib.dq4_gated_fused(ctypes.byref(gate or weight()), ctypes.byref(up or weight()), n_ff, n_in,
                                   dtype, act, x, m, ld_x, h, ld_h, g, u, ld_pre, ws, ws_bytes, None)
    assert call(m=0) == dq4.DQ4_OK
    assert call(n_ff=0) == dq4.DQ4_OK
    for k in (dict(act=0), dict(x=None), dict(h=None), dict(g=ONE), dict(u=ONE), dict(ld_x=1), dict(ld_h=63),
              dict(g=ONE, u=ONE, ld_pre=63), dict(up=weight(ptr=None)), dict(gate=weight(nested_absmax=None)),
              dict(ws_bytes=-1)):
        assert call(**k) == dq4.DQ4_EINVAL, k
    assert call(up=weight(blocksize=128)) == dq4.DQ4_EUNSUPPORTED
    assert call(gate=weight(blocksize=0)) == dq4.DQ4_EUNSUPPORTED


def test_gated_backward_validation(lib):
    def call(n_ff=64, n_in=128, dtype=dq4.DQ4_F16, act=dq4.DQ4_ACT_SILU, dh=ONE, m=4, ld_dh=64, g=ONE, u=ONE,
             ld_pre=64, dx=ONE, ld_dx=128, dg=ONE, du=ONE, ld_d=64, ws=ONE, ws_bytes=BIG):
        return lib.dq4_gated_fused_backward(ctypes.byref(weight()), ctypes.byref(weight()), n_ff, n_in, dtype,
                                            act, dh, m, ld_dh, g, u, ld_pre, dx, ld_dx, dg, du, ld_d, ws,
                                            ws_bytes, None)
    assert call(m=0) == dq4.DQ4_OK
    for k in (dict(act=0), dict(dh=None), dict(g=None), dict(u=None), dict(dx=None), dict(dg=None),
              dict(du=None), dict(ld_dh=1), dict(ld_pre=1), dict(ld_d=1), dict(ld_dx=1), dict(ws_bytes=0)):
        assert call(**k) == dq4.DQ4_EINVAL, k


def test_workspace_sizes(lib):
    w, odd = ctypes.byref(weight()), ctypes.byref(weight(packed=17))
    for name, ws in (("linear_fused", (w,)), ("gated_fused", (w, w)), ("linear_fused_backward", (w,))):
        f = getattr(lib, f"dq4_{name}_workspace_bytes")
        for bad in ((0, 64, 4), (64, -1, 4), (64, 64, 0), (1 << 22, 64, 4), (64, 1 << 22, 4), (64, 64, 1 << 22)):
            assert f(*ws, *bad, ONE, 64, 0) == 0
        assert f(*(None for _ in ws), 64, 64, 4, ONE, 64, 0) == 0
        least, most = f(*ws, 1000, 2048, 300, ONE, 2048, 1), f(*ws, 1000, 2048, 300, ONE, 2048, 0)
        assert 0 < least <= most
        # a misaligned matrix takes a padded copy; the forward calls that read
        # the 4-bit weight once for 128 rows lay x out anew from any rows
        most = f(*ws, 1000, 2048, 1100, ONE, 2048, 0)
        assert f(*ws, 1000, 2048, 1100, P(2), 2048, 0) >= most + 1100 * 1000 * 2
        most = f(*ws, 4096, 4096, 512, ONE, 4096, 0)
        copy = 512 * 4096 * 2 if name.endswith("backward") else 0
        assert f(*ws, 4096, 4096, 512, P(2), 4096, 0) == most + copy
    # one token: the weight is decoded in registers, unless its rows start off a dword
    assert lib.dq4_linear_fused_workspace_bytes(w, 1000, 2048, 1, ONE, 2048, 0) == 0
    assert lib.dq4_linear_fused_workspace_bytes(odd, 1000, 2048, 1, ONE, 2048, 1) > 0
    assert lib.dq4_linear_fused_workspace_bytes(w, 1000, 2047, 1, ONE, 2047, 1) > 0
    assert lib.dq4_gated_fused_workspace_bytes(w, w, 1000, 2048, 1, ONE, 2048, 0) == 0
    assert lib.dq4_gated_fused_workspace_bytes(w, odd, 1000, 2048, 1, ONE, 2048, 1) > 0
    f = lib.dq4_gated_fused_backward_workspace_bytes
    most = f(w, w, 1000, 2048, 300, ONE, ONE, 1000, 0)
    assert 0 < f(w, w, 1000, 2048, 300, ONE, ONE, 1000, 1) <= most
    assert f(w, w, 1000, 2048, 300, ONE, P(2), 1000, 0) >= most + 2 * 300 * 1000 * 2
    assert f(w, w, 0, 64, 4, ONE, ONE, 64, 0) == 0
    # nothing overflows at the largest sizes
    big = 1 << 21
    assert lib.dq4_linear_fused_workspace_bytes(w, big, big, big, P(2), big, 0) == 0
    assert lib.dq4_linear_fused_workspace_bytes(w, big, big, 1 << 18, P(2), big, 0) > 8 << 40


def test_binding_rejects_host_tensors(lib):
    torch = pytest.importorskip("torch")
    u8, f = torch.zeros(4096, dtype=torch.uint8), torch.zeros(256)
    w = dict(packed=u8, scale_codes=u8, nested_absmax=f, scale_codebook=f, codebook4=f[:16], offset=0.0)
    x = torch.zeros((2, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        dq4.dq4_linear_fused(**w, n_out=64, n_in=64, blocksize=64, x=x)
    with pytest.raises(ValueError):
        dq4.dq4_linear_fused_backward(**w, n_out=64, n_in=64, blocksize=64, dy=x)
    with pytest.raises(ValueError):
        dq4.dq4_gated_fused(w, w, 64, 64, 64, x)
    with pytest.raises(ValueError):
        dq4.dq4_gated_fused_backward(w, w, 64, 64, 64, x, x, x)


def test_overlap_of_interleaved_views():
    torch = pytest.importorskip("torch")
    both = torch.zeros((5, 21), dtype=torch.float16)
    a, b, c = both[:, :10], both[:, 10:20], both[:, 9:19]
    assert not dq4._overlap(a, b) and not dq4._overlap(b, a)
    assert dq4._overlap(a, c) and dq4._overlap(c, b) and dq4._overlap(a, a)
    assert not dq4._overlap(a, torch.zeros_like(a)) and not dq4._overlap(a, None)
    assert dq4._overlap(both[1:3], both[2:4]) and not dq4._overlap(both[:2], both[2:])
    flat = torch.zeros(40)
    assert dq4._overlap(flat.as_strided((4, 4), (4, 1)), flat.as_strided((4, 4), (6, 1)))
