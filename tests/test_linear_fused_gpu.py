"""GPU checks of the fused linear and gated calls and their backward passes
against float64 references (bounds: linear_cases.py), and of what the calls
promise about strides, workspaces, streams, graphs and untouched memory."""
from __future__ import annotations

import threading

import numpy as np
import pytest

import block_wise_bit_amd as dq4
from block_wise_bit_amd import inputs
from sum_bounds import U32, gamma_deterministic

torch = pytest.importorskip("torch")

import linear_cases as lc  # noqa: E402
from gpu_util import assert_bits_equal, bits_of  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


def make_weight(n_out, n_in, blocksize=64, fmt="nf4", offset=0.03, seed=0):
    """(host inputs, the binding's keyword arguments with the offset)."""
    x = inputs.make_inputs(n_out * n_in, blocksize, fmt, offset, seed=seed, n_rows=n_out, n_cols=n_in)
    return x, dict(dq4.to_device(x), offset=float(x.offset))


def normal(rng, shape, dt, scale=1.0):
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32))
    return t.to(lc.TYPES[dt][0]).cuda()


# (m, n_out, n_in, blocksize, format): one token and one element upwards, tiles
# met exactly and missed by one on every side, rows that start inside a byte, a
# block and a 16-byte piece, weights of less than one tile
SHAPES = [
    (1, 1, 1, 32, "nf4"), (1, 1, 4096, 64, "nf4"), (5, 3, 7, 32, "fp4"), (2, 127, 65, 32, "nf4"),
    (17, 129, 64, 64, "nf4"), (1, 4096, 4096, 64, "nf4"), (16, 512, 2048, 128, "fp4"),
    (1, 1000, 2376, 64, "nf4"), (37, 1000, 2376, 64, "nf4"), (63, 200, 1032, 256, "nf4"),
    (64, 256, 1024, 4096, "fp4"), (65, 257, 1025, 64, "nf4"), (150, 1001, 1377, 128, "nf4"),
    (256, 512, 512, 64, "nf4"), (257, 640, 520, 32, "fp4"), (300, 1536, 1000, 64, "nf4"),
    (1100, 2176, 352, 64, "nf4"),
    # one to four rows: chunks of 2048 k met, missed and more than the waves;
    # more weight rows than one pass through LDS
    (1, 300, 2048, 64, "nf4"), (2, 70, 2080, 32, "nf4"), (3, 20, 34016, 4096, "fp4"),
    (4, 530, 4128, 64, "nf4"), (1, 9000, 32, 32, "fp4"), (2, 20000, 96, 32, "nf4"),
    (4, 6, 66560, 128, "nf4"), (1, 5, 66560, 64, "nf4"), (3, 257, 6176, 1024, "nf4"),
    # five to 64: chunks of 512 k, rows and columns past the last fragment, more
    # row blocks than workgroups
    (5, 33, 512, 64, "nf4"), (16, 47, 544, 32, "fp4"), (17, 8200, 160, 64, "nf4"),
    (31, 100, 1056, 4096, "nf4"), (33, 4100, 640, 128, "fp4"), (64, 31, 4608, 64, "nf4"),
    (48, 17, 32, 32, "nf4"), (8, 300, 2080, 256, "nf4"), (100, 90, 576, 64, "nf4"),
    (128, 1030, 64, 64, "fp4"), (130, 40, 1056, 32, "nf4"), (192, 300, 512, 64, "nf4"),
    # gradients of few rows: steps of 32 weight rows over all splits, columns
    # and rows that end inside a group or a step
    (1, 3000, 136, 64, "nf4"), (16, 33, 4104, 32, "fp4"), (33, 1025, 264, 4096, "nf4"), (64, 2050, 520, 64, "nf4"),
    # ... with rows of whole dwords only
    (3, 50, 2056, 32, "nf4"), (40, 4200, 168, 64, "nf4"), (20, 90, 1000, 4096, "fp4"),
    # tiles of 128 rows: rows, weight rows and chunks past the last tile, splits
    # that divide the chunks unevenly, more tiles than workgroups
    (65, 300, 1056, 32, "nf4"), (129, 2000, 4128, 64, "fp4"), (600, 33, 544, 64, "nf4"),
    (1024, 700, 2048, 4096, "nf4"), (385, 257, 6176, 256, "nf4"), (900, 20000, 64, 32, "nf4"),
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_forward(shape, dt):
    m, n_out, n_in, bs, fmt = shape
    act = (["none"] + ACTS)[(m + n_out) % 5]
    print(f"linear forward {shape} {dt} {act}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m + n_out))
    host, w = make_weight(n_out, n_in, bs, fmt, seed=n_in)
    x, bias, residual = normal(rng, (m, n_in), dt), normal(rng, (n_out,), dt), normal(rng, (m, n_out), dt)
    pre = torch.full((m, n_out), float("nan"), dtype=x.dtype, device="cuda")
    kw = dict(n_out=n_out, n_in=n_in, blocksize=bs, x=x)
    y = dq4.dq4_linear_fused(**w, **kw, bias=bias, residual=residual, activation=act, pre=pre)
    w64 = lc.weight64(host, dt)
    (z, bz), (ye, by) = lc.linear_expected(dt, act, lc.to64(x), w64, lc.to64(bias), lc.to64(residual))
    lc.check(pre, z, bz, "pre")
    lc.check(y, ye, by, "y")
    plain = dq4.dq4_linear_fused(**w, **kw)
    (z, bz), _ = lc.linear_expected(dt, "none", lc.to64(x), w64)
    lc.check(plain, z, bz, "x W^T")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_forward(shape, dt):
    m, n_ff, n_in, bs, fmt = shape
    act = ACTS[(m + n_ff) % 4]
    print(f"gated forward {shape} {dt} {act}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m + n_ff + 1))
    hg, gate = make_weight(n_ff, n_in, bs, fmt, seed=n_in + 1)
    hu, up = make_weight(n_ff, n_in, bs, fmt, offset=-0.02, seed=n_in + 2)
    x = normal(rng, (m, n_in), dt)
    pre = torch.full((2, m, n_ff), float("nan"), dtype=x.dtype, device="cuda")
    h = dq4.dq4_gated_fused(gate, up, n_ff, n_in, bs, x, activation=act, gate_pre=pre[0], up_pre=pre[1])
    (g, bg), (u, bu), (he, bh) = lc.gated_expected(dt, act, lc.to64(x), lc.weight64(hg, dt),
                                                   lc.weight64(hu, dt))
    lc.check(pre[0], g, bg, "gate_pre")
    lc.check(pre[1], u, bu, "up_pre")
    lc.check(h, he, bh, "h")
    again = dq4.dq4_gated_fused(gate, up, n_ff, n_in, bs, x, activation=act)
    assert_bits_equal(bits_of(again), bits_of(h), "without the pre-activations")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_backward(shape, dt):
    m, n_out, n_in, bs, fmt = shape
    act = (["none"] + ACTS)[(m + n_out + 2) % 5]
    print(f"linear backward {shape} {dt} {act}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m + n_out + 3))
    host, w = make_weight(n_out, n_in, bs, fmt, seed=n_in + 3)
    dy, pre = normal(rng, (m, n_out), dt), normal(rng, (m, n_out), dt, 2.0)
    dx, dz, dbias = dq4.dq4_linear_fused_backward(
        **w, n_out=n_out, n_in=n_in, blocksize=bs, dy=dy, pre=pre, activation=act, bias_grad=True)
    check_linear_backward(dt, act, dy, pre, dx, dz, dbias, lc.weight64(host, dt))
    if act == "none":
        assert dz is dy


def check_linear_backward(dt, act, dy, pre, dx, dz, dbias, w64):
    exact, e, bound = lc.slope_product_expected(dt, act, lc.to64(dy), lc.to64(pre))
    lc.check(dz, exact, bound, "dz")
    # the products' own input is the rounded dz
    got = lc.to64(dz)
    dxe, be = got @ w64, gamma_deterministic(got.shape[1]) * (np.abs(got) @ np.abs(w64))
    lc.check(dx, dxe, lc.rounding(dt, dxe, be), "dx")
    if dbias is not None:
        gm = gamma_deterministic(exact.shape[0])
        lc.check(dbias, exact.sum(0), e.sum(0) * (1 + gm) + gm * np.abs(exact).sum(0) + 1e-37, "dbias")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_backward(shape, dt):
    m, n_ff, n_in, bs, fmt = shape
    act = ACTS[(m + n_ff + 1) % 4]
    print(f"gated backward {shape} {dt} {act}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m + n_ff + 4))
    hg, gate = make_weight(n_ff, n_in, bs, fmt, seed=n_in + 4)
    hu, up = make_weight(n_ff, n_in, bs, fmt, offset=-0.02, seed=n_in + 5)
    dh, g, u = (normal(rng, (m, n_ff), dt, s) for s in (1.0, 2.0, 2.0))
    dx, dgate, dup = dq4.dq4_gated_fused_backward(gate, up, n_ff, n_in, bs, dh, g, u, activation=act)
    dh64, g64, u64 = lc.to64(dh), lc.to64(g), lc.to64(u)
    exact, _, bound = lc.slope_product_expected(dt, act, dh64, g64, u64)
    lc.check(dgate, exact, bound, "dgate")
    exact, bound = lc.value_product_expected(dt, act, dh64, g64)
    lc.check(dup, exact, bound, "dup")
    dg64, du64 = lc.to64(dgate), lc.to64(dup)
    wg, wu = lc.weight64(hg, dt), lc.weight64(hu, dt)
    s = np.abs(dg64) @ np.abs(wg) + np.abs(du64) @ np.abs(wu)
    dxe = dg64 @ wg + du64 @ wu
    lc.check(dx, dxe, lc.rounding(dt, dxe, gamma_deterministic(2 * n_ff) * s), "dx")


# large tiles of the product, whole and split sums, rows and columns that end
# inside a tile: references in float64 on the GPU
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("m,n_out,n_in", [(2000, 8200, 520), (2048, 4096, 11008), (700, 4104, 8200),
                                          (1030, 16500, 136), (520, 2050, 16424),
                                          # a round of whole tiles and one of split tiles
                                          (1000, 8200, 1056), (513, 28672, 1600)])
def test_large_products(m, n_out, n_in, dt):
    print(f"large {m} {n_out} {n_in} {dt}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m))
    tdt, u, sub = lc.TYPES[dt]
    host, w = make_weight(n_out, n_in, 64, "nf4", seed=m)
    hu, up = make_weight(n_out, n_in, 64, "nf4", offset=-0.02, seed=m + 1)
    w64, wu64 = (torch.from_numpy(lc.weight64(h, dt)).cuda() for h in (host, hu))

    def close(got, exact, s, k, what):
        gamma = gamma_deterministic(k)
        err = (got.double() - exact).abs()
        bound = gamma * s + u * (exact.abs() + gamma * s) + sub
        print(f"{what}: worst err/bound {float((err / bound).max()):.3f}", flush=True)
        assert bool(torch.isfinite(got).all()) and bool((err <= bound).all()), what
    x, dy = normal(rng, (m, n_in), dt), normal(rng, (m, n_out), dt)
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)
    y = dq4.dq4_linear_fused(**w, **sizes, x=x)
    close(y, x.double() @ w64.t(), x.double().abs() @ w64.abs().t(), n_in, "forward")
    dx, _, _ = dq4.dq4_linear_fused_backward(**w, **sizes, dy=dy)
    close(dx, dy.double() @ w64, dy.double().abs() @ w64.abs(), n_out, "backward")
    pre = torch.empty((2, m, n_out), dtype=tdt, device="cuda")
    h = dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x, activation="relu", gate_pre=pre[0], up_pre=pre[1])
    close(pre[0], x.double() @ w64.t(), x.double().abs() @ w64.abs().t(), n_in, "gate_pre")
    close(pre[1], x.double() @ wu64.t(), x.double().abs() @ wu64.abs().t(), n_in, "up_pre")
    dx, dg, du = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, dy, pre[0], pre[1], activation="relu")
    close(dx, dg.double() @ w64 + du.double() @ wu64, dg.double().abs() @ w64.abs() + du.double().abs() @ wu64.abs(),
          2 * n_out, "gated backward")


# ----------------------------------------------------------------------------
# strides, neighbours and windows
# ----------------------------------------------------------------------------
def padded(t, left, right, below, fill=float("nan")):
    """(the buffer, t's values as a strided view inside it)."""
    m, n = t.shape
    big = torch.full((m + below, left + n + right), fill, dtype=t.dtype, device=t.device)
    view = big[:m, left:left + n]
    view.copy_(t)
    return big, view


def untouched(big, view_shape, left, fill):
    m, n = view_shape
    keep = torch.ones_like(big, dtype=torch.bool)
    keep[:m, left:left + n] = False
    assert bool((big[keep] == fill).all()), "memory outside the matrix was written"


@pytest.mark.parametrize("left,right", [(0, 8), (1, 0), (8, 16), (3, 4)])
@pytest.mark.parametrize("m,n_out,n_in", [(1, 264, 512), (5, 264, 512), (3, 264, 2080), (33, 264, 520),
                                          (64, 264, 544), (130, 200, 1001), (200, 264, 1056)])
def test_strided_matrices(m, n_out, n_in, left, right):
    """Every matrix inside a larger buffer: NaN around the inputs, a mark around
    the outputs; the results equal the dense call's bit for bit."""
    rng = np.random.Generator(np.random.PCG64(m + left))
    _, w = make_weight(n_out, n_in, seed=9)
    _, up = make_weight(n_out, n_in, seed=10)
    x, bias, res = normal(rng, (m, n_in), "bf16"), normal(rng, (n_out,), "bf16"), normal(rng, (m, n_out), "bf16")
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)
    mark = 777.0

    def out(width):
        return padded(torch.zeros((m, width), dtype=torch.bfloat16, device="cuda"), left, right, 2, mark)

    def inp(t):
        return padded(t, left, right, 2)[1]
    pre = torch.empty_like(res)
    y = dq4.dq4_linear_fused(**w, **sizes, x=x, bias=bias, residual=res, activation="silu", pre=pre)
    big_y, ys = out(n_out)
    big_p, ps = out(n_out)
    dq4.dq4_linear_fused(**w, **sizes, x=inp(x), bias=bias, residual=inp(res), activation="silu", y=ys, pre=ps)
    assert_bits_equal(bits_of(ys.contiguous()), bits_of(y), "y")
    assert_bits_equal(bits_of(ps.contiguous()), bits_of(pre), "pre")
    untouched(big_y, (m, n_out), left, mark)
    untouched(big_p, (m, n_out), left, mark)

    g, u = torch.empty_like(res), torch.empty_like(res)
    h = dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x, gate_pre=g, up_pre=u)
    big_h, hs = out(n_out)
    both = torch.full((m + 1, 2 * n_out + 3), mark, dtype=torch.bfloat16, device="cuda")
    gs, us = both[:m, 1:1 + n_out], both[:m, 1 + n_out:1 + 2 * n_out]   # interleaved halves
    dq4.dq4_gated_fused(w, up, n_out, n_in, 64, inp(x), h=hs, gate_pre=gs, up_pre=us)
    for a, b in ((hs, h), (gs, g), (us, u)):
        assert_bits_equal(bits_of(a.contiguous()), bits_of(b), "gated")
    untouched(big_h, (m, n_out), left, mark)
    untouched(both, (m, 2 * n_out), 1, mark)

    dx, dz, db = dq4.dq4_linear_fused_backward(**w, **sizes, dy=res, pre=pre, activation="gelu", bias_grad=True)
    big_x, xs = out(n_in)
    big_z, zs = out(n_out)
    _, _, db2 = dq4.dq4_linear_fused_backward(**w, **sizes, dy=inp(res), pre=inp(pre), activation="gelu",
                                              bias_grad=True, dx=xs, dz=zs)
    for a, b in ((xs, dx), (zs, dz)):
        assert_bits_equal(bits_of(a.contiguous()), bits_of(b), "linear backward")
    assert_bits_equal(bits_of(db2), bits_of(db), "dbias")
    untouched(big_x, (m, n_in), left, mark)
    untouched(big_z, (m, n_out), left, mark)
    dx, _, _ = dq4.dq4_linear_fused_backward(**w, **sizes, dy=res)
    dq4.dq4_linear_fused_backward(**w, **sizes, dy=inp(res), dx=xs)
    assert_bits_equal(bits_of(xs.contiguous()), bits_of(dx), "dx without activation")

    dx, dg, du = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, res, g, u)
    both.fill_(mark)
    dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, inp(res), inp(g), inp(u), dx=xs, dgate=gs, dup=us)
    for a, b in ((xs, dx), (gs, dg), (us, du)):
        assert_bits_equal(bits_of(a.contiguous()), bits_of(b), "gated backward")
    untouched(both, (m, 2 * n_out), 1, mark)
    untouched(big_x, (m, n_in), left, mark)


@pytest.mark.parametrize("m,n_out,n_in", [(3, 700, 515), (3, 768, 512), (20, 768, 512), (200, 768, 512),
                                          (200, 4096, 2048)])
def test_any_workspace_gives_the_same_bits(m, n_out, n_in):
    """The least workspace (windows of output columns), one in between, and
    one full of NaN."""
    rng = np.random.Generator(np.random.PCG64(5))
    _, w = make_weight(n_out, n_in, seed=11)
    _, up = make_weight(n_out, n_in, seed=12)
    x, dy = normal(rng, (m, n_in), "f16"), normal(rng, (m, n_out), "f16")
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)

    def buffers(size, *args):
        least, most = size(n_out, n_in, m, *args, least=True), size(n_out, n_in, m, *args)
        assert least <= most
        for n in (least, (least + most) // 2, most, most + 1000):
            yield torch.full((n // 2 + 1,), float("nan"), dtype=torch.float16, device="cuda").view(torch.uint8)[:n]
    y = dq4.dq4_linear_fused(**w, **sizes, x=x)
    for ws in buffers(dq4.dq4_linear_fused_workspace_bytes, x):
        assert_bits_equal(bits_of(dq4.dq4_linear_fused(**w, **sizes, x=x, workspace=ws)), bits_of(y), "y")
    h = dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x)
    for ws in buffers(dq4.dq4_gated_fused_workspace_bytes, x):
        assert_bits_equal(bits_of(dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x, workspace=ws)), bits_of(h), "h")
    dx, _, db = dq4.dq4_linear_fused_backward(**w, **sizes, dy=dy, bias_grad=True)
    for ws in buffers(dq4.dq4_linear_fused_backward_workspace_bytes, dy):
        got = dq4.dq4_linear_fused_backward(**w, **sizes, dy=dy, bias_grad=True, workspace=ws)
        assert_bits_equal(bits_of(got[0]), bits_of(dx), "dx")
        assert_bits_equal(bits_of(got[2]), bits_of(db), "dbias")
    g, u = normal(rng, (m, n_out), "f16"), normal(rng, (m, n_out), "f16")
    dx = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, dy, g, u)[0]
    for ws in buffers(dq4.dq4_gated_fused_backward_workspace_bytes):
        got = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, dy, g, u, workspace=ws)
        assert_bits_equal(bits_of(got[0]), bits_of(dx), "dx")
    torch.cuda.synchronize()


@pytest.mark.parametrize("m", [1, 9, 200])
def test_residual_in_place(m):
    rng = np.random.Generator(np.random.PCG64(m))
    _, w = make_weight(384, 512, seed=13)
    x, res = normal(rng, (m, 512), "bf16"), normal(rng, (m, 384), "bf16")
    sizes = dict(n_out=384, n_in=512, blocksize=64)
    want = dq4.dq4_linear_fused(**w, **sizes, x=x, residual=res)
    got = dq4.dq4_linear_fused(**w, **sizes, x=x, residual=res, y=res)
    assert got is res
    assert_bits_equal(bits_of(res), bits_of(want), "y over its residual")


def test_unaligned_codes_and_single_row_strides():
    """Packed codes that start on an odd byte (another kernel then, another
    order of the sums); a single row whose stride is nonsense (torch leaves it
    so)."""
    rng = np.random.Generator(np.random.PCG64(21))
    for m in (1, 70):
        host, w = make_weight(256, 512, seed=14)
        w64 = lc.weight64(host, "bf16")
        x, dy = normal(rng, (m, 512), "bf16"), normal(rng, (m, 256), "bf16")
        odd = torch.empty(w["packed"].numel() + 1, dtype=torch.uint8, device="cuda")
        odd[1:] = w["packed"]
        w1 = dict(w, packed=odd[1:])
        y = dq4.dq4_linear_fused(**w1, n_out=256, n_in=512, blocksize=64, x=x)
        (z, bz), _ = lc.linear_expected("bf16", "none", lc.to64(x), w64)
        lc.check(y, z, bz, "odd codes, forward")
        dx, dz, _ = dq4.dq4_linear_fused_backward(**w1, n_out=256, n_in=512, blocksize=64, dy=dy)
        check_linear_backward("bf16", "none", dy, dy, dx, dz, None, w64)
    row = torch.as_strided(x[:1].contiguous(), (1, 512), (1, 1))
    y1 = dq4.dq4_linear_fused(**w, n_out=256, n_in=512, blocksize=64, x=row)
    assert_bits_equal(bits_of(y1), bits_of(dq4.dq4_linear_fused(**w, n_out=256, n_in=512, blocksize=64,
                                                                x=x[:1].contiguous())), "single row")


@pytest.mark.parametrize("m,n_in", [(2, 2080), (4, 96), (20, 544), (20, 520), (90, 96)])
def test_values_that_no_code_uses(m, n_in):
    """Infinities and NaN in the codebooks reach the elements whose codes name
    them, and nothing that lies beyond a row or in the padding."""
    rng = np.random.Generator(np.random.PCG64(23))
    host, w = make_weight(48, n_in, seed=20)
    # code 0 (what a load beyond the weight gives) and scale code 0 are unused
    packed = torch.where((w["packed"] & 15) == 0, w["packed"] | 1, w["packed"])
    packed = torch.where((packed >> 4) == 0, packed | 16, packed)
    codes = torch.clamp(w["scale_codes"], min=1)
    plain = dict(w, packed=packed, scale_codes=codes)
    bad = dict(plain, codebook4=w["codebook4"].clone(), scale_codebook=w["scale_codebook"].clone())
    bad["codebook4"][0] = float("inf")
    bad["scale_codebook"][0] = float("nan")
    x = normal(rng, (m, n_in), "bf16")
    dy = normal(rng, (m, 48), "bf16")
    for a, b in ((dq4.dq4_linear_fused(**t, n_out=48, n_in=n_in, blocksize=64, x=x) for t in (plain, bad)),
                 (dq4.dq4_gated_fused(t, t, 48, n_in, 64, x) for t in (plain, bad)),
                 (dq4.dq4_linear_fused_backward(**t, n_out=48, n_in=n_in, blocksize=64, dy=dy)[0]
                  for t in (plain, bad))):
        assert_bits_equal(bits_of(b), bits_of(a), "unused codebook entries")


def test_rows_do_not_mix():
    """A row of NaN or infinities reaches its own outputs only."""
    rng = np.random.Generator(np.random.PCG64(22))
    _, w = make_weight(300, 520, seed=15)
    _, up = make_weight(300, 520, seed=16)
    for m in (6, 40, 90):
        x = normal(rng, (m, 520), "bf16")
        bad = x.clone()
        bad[2] = float("nan")
        bad[4, 7] = float("inf")
        others = [r for r in range(m) if r not in (2, 4)]
        y, yb = (dq4.dq4_linear_fused(**w, n_out=300, n_in=520, blocksize=64, x=t) for t in (x, bad))
        assert_bits_equal(bits_of(yb[others]), bits_of(y[others]), "linear")
        assert bool(torch.isnan(yb[2]).all()) and not bool(torch.isfinite(yb[4]).all())
        h, hb = (dq4.dq4_gated_fused(w, up, 300, 520, 64, t) for t in (x, bad))
        assert_bits_equal(bits_of(hb[others]), bits_of(h[others]), "gated")
        dx, dxb = (dq4.dq4_linear_fused_backward(**w, n_out=300, n_in=520, blocksize=64, dy=t[:, :300].contiguous())[0]
                   for t in (x, bad))
        assert_bits_equal(bits_of(dxb[others]), bits_of(dx[others]), "backward")
        assert bool(torch.isnan(dxb[2]).all())


def test_extreme_pre_activations():
    """The slopes at the ends of the type's range: 0 and 1, never NaN."""
    for dt in ("f16", "bf16"):
        tdt = lc.TYPES[dt][0]
        big = torch.finfo(tdt).max
        vals = torch.tensor([-big, -200.0, -90.0, -0.0, 0.0, 90.0, 200.0, big], dtype=torch.float32)
        pre = vals.repeat(8).view(1, 64).to(tdt).cuda()
        dy = torch.ones_like(pre)
        _, w = make_weight(64, 64, seed=17)
        for act in ACTS:
            _, dz, _ = dq4.dq4_linear_fused_backward(**w, n_out=64, n_in=64, blocksize=64, dy=dy, pre=pre,
                                                     activation=act)
            half = 0.0 if act == "relu" else 0.5
            want = torch.tensor([0, 0, 0, half, half, 1, 1, 1], dtype=torch.float32)
            assert torch.equal(dz.float().cpu()[0, :8], want), (dt, act, dz[0, :8])


def test_empty_sizes():
    host, w = make_weight(64, 128, seed=18)
    e = dict(blocksize=64)
    x = torch.zeros((0, 128), dtype=torch.float16, device="cuda")
    assert dq4.dq4_linear_fused(**w, n_out=64, n_in=128, x=x, **e).shape == (0, 64)
    assert dq4.dq4_gated_fused(w, w, 64, 128, 64, x).shape == (0, 64)
    dx, dz, db = dq4.dq4_linear_fused_backward(**w, n_out=64, n_in=128, dy=x[:, :64].contiguous(), bias_grad=True, **e)
    assert dx.shape == (0, 128) and bool((db == 0).all())
    dx, dg, du = dq4.dq4_gated_fused_backward(w, w, 64, 128, 64, x[:, :64].contiguous(), x[:, :64].contiguous(),
                                              x[:, :64].contiguous())
    assert dx.shape == (0, 128) and dg.shape == (0, 64)
    # empty sums: no input columns, no output columns
    for m in (2, 100):
        none = torch.zeros((m, 0), dtype=torch.float16, device="cuda")
        bias = torch.arange(64, dtype=torch.float16, device="cuda")
        y = dq4.dq4_linear_fused(**w, n_out=64, n_in=0, x=none, bias=bias, **e)
        assert torch.equal(y, bias.expand(m, 64))
        assert bool((dq4.dq4_gated_fused(w, w, 64, 0, 64, none) == 0).all())
        dx, dz, db = dq4.dq4_linear_fused_backward(**w, n_out=0, n_in=128, dy=none, bias_grad=True, **e)
        assert dx.shape == (m, 128) and bool((dx == 0).all()) and db.numel() == 0
        assert bool((dq4.dq4_gated_fused_backward(w, w, 0, 128, 64, none, none, none)[0] == 0).all())
        dx, dz, db = dq4.dq4_linear_fused_backward(**w, n_out=64, n_in=0, dy=torch.ones((m, 64), dtype=torch.float16,
                                                                                        device="cuda"),
                                                   bias_grad=True, **e)
        assert dx.shape == (m, 0) and bool((db == m).all())


# ----------------------------------------------------------------------------
# the block as a model runs it
# ----------------------------------------------------------------------------
def feed_forward(gate, up, down, sizes, x, residual):
    n_ff, n_in, bs = sizes
    pre = torch.empty((2, x.size(0), n_ff), dtype=x.dtype, device="cuda")
    h = dq4.dq4_gated_fused(gate, up, n_ff, n_in, bs, x, gate_pre=pre[0], up_pre=pre[1])
    y = dq4.dq4_linear_fused(**down, n_out=n_in, n_in=n_ff, blocksize=bs, x=h, residual=residual)
    return y, h, pre


@pytest.mark.parametrize("dt,m", [("f16", 1), ("f16", 70), ("bf16", 300)])
def test_feed_forward_block(dt, m):
    """Gated half, down projection onto the residual stream, and back: each
    stage against float64 from the stage before, the input gradient against
    central differences of the float64 block."""
    n_ff, n_in, bs = 688, 256, 64
    sizes = (n_ff, n_in, bs)
    rng = np.random.Generator(np.random.PCG64(31))
    (hg, gate), (hu, up) = make_weight(n_ff, n_in, bs, seed=41), make_weight(n_ff, n_in, bs, seed=42)
    hd, down = make_weight(n_in, n_ff, bs, seed=43)
    x, dy = normal(rng, (m, n_in), dt), normal(rng, (m, n_in), dt)
    y, h, pre = feed_forward(gate, up, down, sizes, x, x)
    wg, wu, wd = (lc.weight64(t, dt) for t in (hg, hu, hd))
    (_, _), (_, _), (he, bh) = lc.gated_expected(dt, "silu", lc.to64(x), wg, wu)
    lc.check(h, he, bh, "h")
    _, (ye, by) = lc.linear_expected(dt, "none", lc.to64(h), wd, None, lc.to64(x))
    lc.check(y, ye, by, "y")
    dh, _, _ = dq4.dq4_linear_fused_backward(**down, n_out=n_in, n_in=n_ff, blocksize=bs, dy=dy)
    dx, dgate, dup = dq4.dq4_gated_fused_backward(gate, up, n_ff, n_in, bs, dh, pre[0], pre[1])
    total = lc.to64(dx) + lc.to64(dy)

    def loss(v):
        g, u = v @ wg.T, v @ wu.T
        return ((lc.act64("silu", g) * u) @ wd.T + v) * lc.to64(dy)
    # directional derivatives along random directions, per row
    x64 = lc.to64(x)
    u_t = lc.TYPES[dt][1]
    # roundings on the way: pre, dh, dgate/dup, dx, each half a step, every one
    # carried through products whose size `scale` bounds by absolute values
    dh_abs = np.abs(lc.to64(dy)) @ np.abs(wd)
    g64, u64 = np.abs(lc.to64(pre[0])), np.abs(lc.to64(pre[1]))
    scale = (dh_abs * (1.1 * u64 + g64 + 1.1 * u64 * (1 + g64))) @ np.abs(wg) + (dh_abs * (1.1 * g64 + g64)) @ np.abs(wu)
    for k in range(3):
        d = np.random.Generator(np.random.PCG64(50 + k)).standard_normal(x64.shape)
        eps = 1e-5
        diff = (loss(x64 + eps * d).sum(1) - loss(x64 - eps * d).sum(1)) / (2 * eps)
        got = (total * d).sum(1)
        bound = 4 * u_t * ((scale + np.abs(total)) * np.abs(d)).sum(1) + 1e-6 * np.abs(diff) + 1e-6
        assert (np.abs(got - diff) <= bound).all(), (got, diff, bound)


@pytest.mark.parametrize("m,n_ff,n_in", [(40, 512, 256), (300, 4096, 2048)])
def test_graph_replays_follow_new_inputs(m, n_ff, n_in):
    """The whole block, forward and backward, captured once and replayed four
    times with new inputs and eager work in between; two graphs share one
    stream and one set of buffers."""
    bs = 64
    rng = np.random.Generator(np.random.PCG64(61))
    gate, up, down = (make_weight(*s, seed=k)[1] for s, k in (((n_ff, n_in), 51), ((n_ff, n_in), 52), ((n_in, n_ff), 53)))
    x, dy = normal(rng, (m, n_in), "bf16"), normal(rng, (m, n_in), "bf16")

    def step(xv, dyv):
        y, h, pre = feed_forward(gate, up, down, (n_ff, n_in, bs), xv, xv)
        dh, _, db = dq4.dq4_linear_fused_backward(**down, n_out=n_in, n_in=n_ff, blocksize=bs, dy=dyv, bias_grad=True)
        return (y,) + dq4.dq4_gated_fused_backward(gate, up, n_ff, n_in, bs, dh, pre[0], pre[1]) + (db,)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, dy)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(x, dy)
        graphs.append((g, outs))
    for rep in range(4):
        x.copy_(normal(rng, (m, n_in), "bf16"))
        dy.copy_(normal(rng, (m, n_in), "bf16"))
        want = step(x, dy)
        torch.cuda.synchronize()
        for g, outs in graphs:
            for t in outs:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert_bits_equal(bits_of(a), bits_of(b), f"replay {rep}")


def test_on_another_stream():
    """Called with stream=: the results are ready in that stream's order."""
    rng = np.random.Generator(np.random.PCG64(71))
    _, w = make_weight(1024, 2048, seed=61)
    side = torch.cuda.Stream()
    for m in (1, 200):
        x = normal(rng, (m, 2048), "bf16")
        sizes = dict(n_out=1024, n_in=2048, blocksize=64)
        want = dq4.dq4_linear_fused(**w, **sizes, x=x)
        back = dq4.dq4_linear_fused_backward(**w, **sizes, dy=want, bias_grad=True)
        torch.cuda.synchronize()
        got = dq4.dq4_linear_fused(**w, **sizes, x=x, stream=side)
        got_back = dq4.dq4_linear_fused_backward(**w, **sizes, dy=got, bias_grad=True, stream=side)
        side.synchronize()
        assert_bits_equal(bits_of(got), bits_of(want), "forward")
        for a, b in zip(got_back, back):
            assert_bits_equal(bits_of(a), bits_of(b), "backward")


def test_two_threads_at_once():
    """Calls from two threads, each on a stream of its own, do not share
    anything: every result has the bits of the call alone."""
    rng = np.random.Generator(np.random.PCG64(72))
    _, w = make_weight(1024, 2048, seed=62)
    _, up = make_weight(1024, 2048, seed=63)
    sizes = dict(n_out=1024, n_in=2048, blocksize=64)
    xs = [normal(rng, (m, 2048), "bf16") for m in (1, 40, 200, 1100)]

    def calls(x):
        h = dq4.dq4_gated_fused(w, up, 1024, 2048, 64, x)
        y = dq4.dq4_linear_fused(**w, **sizes, x=x, bias=h[0].contiguous())
        dx, _, db = dq4.dq4_linear_fused_backward(**w, **sizes, dy=y, bias_grad=True)
        return h, y, dx, db
    want = [calls(x) for x in xs]
    torch.cuda.synchronize()
    got, failed = [{}, {}], []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for rep in range(5):
                    for j in (range(4) if i == 0 else reversed(range(4))):
                        got[i][j] = calls(xs[j])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported by the test's own thread
            failed.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i in range(2):
        for j in range(4):
            for a, b in zip(got[i][j], want[j]):
                assert_bits_equal(bits_of(a), bits_of(b), f"thread {i}")


def test_refusals():
    _, w = make_weight(64, 128, seed=19)
    s = dict(n_out=64, n_in=128, blocksize=64)
    x = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    y = torch.zeros((4, 64), dtype=torch.float16, device="cuda")

    def refused(f, *a, **k):
        with pytest.raises(ValueError):
            f(*a, **k)
    f, b = dq4.dq4_linear_fused, dq4.dq4_linear_fused_backward
    refused(f, **w, **s, x=x.float())
    refused(f, **w, **s, x=x.cpu())
    refused(f, **w, **s, x=x[:, :100])
    refused(f, **w, **s, x=x.t().contiguous().t())                  # column-major rows
    refused(f, **w, **s, x=x[:1].expand(4, 128))                    # row stride 0
    refused(f, **w, **s, x=x, activation="swish")
    refused(f, **w, **s, x=x, bias=torch.zeros(65, dtype=torch.float16, device="cuda"))
    refused(f, **w, **s, x=x, bias=torch.zeros(64, dtype=torch.float32, device="cuda"))
    refused(f, **w, **s, x=x, bias=torch.zeros(128, dtype=torch.float16, device="cuda")[::2])
    refused(f, **w, **s, x=x, residual=y.bfloat16())
    refused(f, **w, **s, x=x, y=y[:3])
    refused(f, **w, **s, x=x, y=x[:, :64])                          # y over x
    refused(f, **w, **s, x=x, y=y, pre=y)
    refused(f, **w, **s, x=x.repeat(100, 1), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(f, **w, **s, x=x.repeat(100, 1), workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[8:])
    refused(f, **w, **dict(s, blocksize=48), x=x)
    refused(f, **w, **dict(s, n_out=65), x=x)                       # more than the weight holds
    refused(f, **w, **dict(s, n_out=-1), x=x)
    refused(f, **w, **s, x=x, nested_blocksize=128)
    refused(b, **w, **s, dy=y, activation="gelu")                   # no pre
    refused(b, **w, **s, dy=y, dz=torch.empty_like(y))              # dz is dy
    refused(b, **w, **s, dy=y, pre=y, activation="gelu", dz=y)      # dz over dy
    refused(b, **w, **s, dy=x)
    refused(b, **w, **s, dy=y, dbias=torch.zeros(64, dtype=torch.float16, device="cuda"))
    g, gb = dq4.dq4_gated_fused, dq4.dq4_gated_fused_backward
    refused(g, w, w, 64, 128, 64, x, activation="none")
    refused(g, w, w, 64, 128, 64, x, gate_pre=y)
    refused(g, w, w, 64, 128, 64, x, gate_pre=y, up_pre=torch.zeros((4, 72), dtype=torch.float16, device="cuda")[:, :64])
    refused(g, w, w, 64, 128, 64, x, gate_pre=y, up_pre=y)
    refused(g, w, {k: v for k, v in w.items() if k != "packed"} | {"packed": w["packed"].cpu()}, 64, 128, 64, x)
    refused(gb, w, w, 64, 128, 64, y, y, y[:3])
    refused(gb, w, w, 64, 128, 64, y, y, y, dgate=y)                # dgate over dh
    torch.cuda.synchronize()
