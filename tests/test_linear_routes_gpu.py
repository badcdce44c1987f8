"""The fused linear and gated calls, kernel by kernel: shapes chosen by the
restated plan (linear_plan.py) so that each kernel and each of its forms is
reached, against float64 references (bounds: linear_cases.py); rows that do not
mix and codes that no element uses, on the kernels with padded operands; and
every element of the weight, read out through one-hot rows, on every kernel that
decodes."""
from __future__ import annotations

import numpy as np
import pytest

import block_wise_bit_amd as dq4

torch = pytest.importorskip("torch")

import linear_cases as lc  # noqa: E402
import linear_plan as plan  # noqa: E402
from gpu_util import assert_bits_equal, bits_of  # noqa: E402
from sum_bounds import gamma_deterministic  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
T = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


@pytest.fixture(autouse=True)
def products_on_the_gpu(monkeypatch):
    """linear_cases' reference product in float64 on the GPU: these are large."""
    def product64(x, w, dt):
        a, b = torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda()
        z, s = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
        return z.cpu().numpy(), gamma_deterministic(max(x.shape[1], 1)) * s.cpu().numpy()
    monkeypatch.setattr(lc, "product64", product64)


def make_weight(n_out, n_in, blocksize, seed, scale=-3.0, offset=0.03):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = n_out * n_in
    blocks = -(-n // blocksize)
    cb4 = torch.sort(torch.rand(16, generator=gen, device="cuda") * 2 - 1).values
    return dict(
        packed=torch.randint(0, 256, (-(-n // 2),), generator=gen, device="cuda", dtype=torch.uint8),
        scale_codes=torch.randint(0, 256, (blocks,), generator=gen, device="cuda", dtype=torch.uint8),
        nested_absmax=torch.exp(torch.randn(-(-blocks // 256), generator=gen, device="cuda") * 0.5 + scale),
        scale_codebook=torch.sort(torch.rand(256, generator=gen, device="cuda") * 2 - 1).values,
        codebook4=cb4, offset=offset)


def weight_values(w, n_out, n_in, blocksize, dt):
    """W as the dequantization writes it (bit-exact against the oracle: the
    tests of dq4_nested_dequant)."""
    return dq4.dq4_nested_dequant(**w, n=n_out * n_in, blocksize=blocksize, out_dtype=T[dt]).view(n_out, n_in)


def normal(seed, shape, dt, scale=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(T[dt])


# ----------------------------------------------------------------------------
# the 128-row tiles
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("i", range(len(plan.TILE_LINEAR)))
def test_tiles_linear(i):
    m, n_out, n_in, bs = plan.TILE_LINEAR[i]
    dt, act = ("bf16", "f16")[i % 2], (["none"] + ACTS)[i % 5]
    print(f"tiles linear {m} {n_out} {n_in} {bs} {dt} {act} {plan.tile_kind(m, n_out, n_in, bs, False)}", flush=True)
    w = make_weight(n_out, n_in, bs, i)
    x, bias, res = normal(1, (m, n_in), dt), normal(2, (n_out,), dt), normal(3, (m, n_out), dt)
    pre = torch.full((m, n_out), float("nan"), dtype=x.dtype, device="cuda")
    y = dq4.dq4_linear_fused(**w, n_out=n_out, n_in=n_in, blocksize=bs, x=x, bias=bias, residual=res, activation=act,
                             pre=pre)
    w64 = lc.to64(weight_values(w, n_out, n_in, bs, dt))
    (z, bz), (ye, by) = lc.linear_expected(dt, act, lc.to64(x), w64, lc.to64(bias), lc.to64(res))
    lc.check(pre, z, bz, "pre")
    lc.check(y, ye, by, "y")


@pytest.mark.parametrize("i", range(len(plan.TILE_GATED)))
def test_tiles_gated(i):
    m, n_ff, n_in, bs = plan.TILE_GATED[i]
    dt, act = ("f16", "bf16")[i % 2], ACTS[i % 4]
    print(f"tiles gated {m} {n_ff} {n_in} {bs} {dt} {act} {plan.tile_kind(m, n_ff, n_in, bs, True)}", flush=True)
    gate, up = make_weight(n_ff, n_in, bs, i + 20), make_weight(n_ff, n_in, bs, i + 40, offset=-0.02)
    x = normal(4, (m, n_in), dt)
    pre = torch.full((2, m, n_ff), float("nan"), dtype=x.dtype, device="cuda")
    h = dq4.dq4_gated_fused(gate, up, n_ff, n_in, bs, x, activation=act, gate_pre=pre[0], up_pre=pre[1])
    wg, wu = (lc.to64(weight_values(t, n_ff, n_in, bs, dt)) for t in (gate, up))
    (g, bg), (u, bu), (he, bh) = lc.gated_expected(dt, act, lc.to64(x), wg, wu)
    lc.check(pre[0], g, bg, "gate_pre")
    lc.check(pre[1], u, bu, "up_pre")
    lc.check(h, he, bh, "h")


@pytest.mark.parametrize("left,right", [(0, 8), (3, 4)])
@pytest.mark.parametrize("gated,shape", [(False, plan.TILE_LINEAR[0]), (False, plan.TILE_LINEAR[5]),
                                         (True, plan.TILE_GATED[0]), (True, plan.TILE_GATED[5])])
def test_tiles_in_strided_matrices(gated, shape, left, right):
    """Inputs inside NaN, outputs inside marked buffers, 16-byte aligned or
    not: the dense call's bits, and nothing else written."""
    m, n_out, n_in, bs = shape
    assert plan.forward_route(m, n_out, n_in, gated) == "tile"
    mark = 777.0

    def put(t, fill):
        big = torch.full((t.size(0) + 2, left + t.size(1) + right), fill, dtype=t.dtype, device="cuda")
        view = big[:t.size(0), left:left + t.size(1)]
        view.copy_(t)
        return big, view

    def untouched(big, view):
        inside = torch.zeros_like(big, dtype=torch.bool)
        inside[:view.size(0), left:left + view.size(1)] = True
        assert bool((big[~inside] == mark).all())
    w, up = make_weight(n_out, n_in, bs, 60), make_weight(n_out, n_in, bs, 61)
    x, bias, res = normal(5, (m, n_in), "bf16"), normal(6, (n_out,), "bf16"), normal(7, (m, n_out), "bf16")
    _, xs = put(x, float("nan"))
    outs = [put(torch.zeros_like(res), mark) for _ in range(3)]
    if gated:
        want = [torch.empty_like(res) for _ in range(3)]
        dq4.dq4_gated_fused(w, up, n_out, n_in, bs, x, h=want[0], gate_pre=want[1], up_pre=want[2])
        dq4.dq4_gated_fused(w, up, n_out, n_in, bs, xs, h=outs[0][1], gate_pre=outs[1][1], up_pre=outs[2][1])
    else:
        sizes = dict(n_out=n_out, n_in=n_in, blocksize=bs, bias=bias, activation="silu")
        want = [torch.empty_like(res) for _ in range(2)]
        dq4.dq4_linear_fused(**w, **sizes, x=x, residual=res, y=want[0], pre=want[1])
        dq4.dq4_linear_fused(**w, **sizes, x=xs, residual=put(res, float("nan"))[1], y=outs[0][1], pre=outs[1][1])
    for (big, view), t in zip(outs, want):
        assert_bits_equal(bits_of(view.contiguous()), bits_of(t), "strided")
        untouched(big, view)


# ----------------------------------------------------------------------------
# the product's tiles (odd widths)
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("i", range(len(plan.PRODUCTS)))
def test_products_forward(i):
    m, n_out, n_in = plan.PRODUCTS[i]
    dt, act = ("f16", "bf16")[i % 2], (["none"] + ACTS)[i % 5]
    assert plan.forward_route(m, n_out, n_in, False) == "product"
    print(f"product {m} {n_out} {n_in} {dt} {act}", flush=True)
    w = make_weight(n_out, n_in, 64, i + 70)
    x, bias, res = normal(8, (m, n_in), dt), normal(9, (n_out,), dt), normal(10, (m, n_out), dt)
    pre = torch.full((m, n_out), float("nan"), dtype=x.dtype, device="cuda")
    y = dq4.dq4_linear_fused(**w, n_out=n_out, n_in=n_in, blocksize=64, x=x, bias=bias, residual=res, activation=act,
                             pre=pre)
    w64 = lc.to64(weight_values(w, n_out, n_in, 64, dt))
    (z, bz), (ye, by) = lc.linear_expected(dt, act, lc.to64(x), w64, lc.to64(bias), lc.to64(res))
    lc.check(pre, z, bz, "pre")
    lc.check(y, ye, by, "y")


@pytest.mark.parametrize("i", range(len(plan.PRODUCTS_GATED)))
def test_products_gated(i):
    m, n_ff, n_in = plan.PRODUCTS_GATED[i]
    dt, act = ("bf16", "f16")[i % 2], ACTS[i % 4]
    assert plan.forward_route(m, n_ff, n_in, True) == "product"
    print(f"gated product {m} {n_ff} {n_in} {dt} {act}", flush=True)
    gate, up = make_weight(n_ff, n_in, 64, i + 80), make_weight(n_ff, n_in, 64, i + 90)
    x = normal(11, (m, n_in), dt)
    pre = torch.full((2, m, n_ff), float("nan"), dtype=x.dtype, device="cuda")
    h = dq4.dq4_gated_fused(gate, up, n_ff, n_in, 64, x, activation=act, gate_pre=pre[0], up_pre=pre[1])
    wg, wu = (lc.to64(weight_values(t, n_ff, n_in, 64, dt)) for t in (gate, up))
    (g, bg), (u, bu), (he, bh) = lc.gated_expected(dt, act, lc.to64(x), wg, wu)
    lc.check(pre[0], g, bg, "gate_pre")
    lc.check(pre[1], u, bu, "up_pre")
    lc.check(h, he, bh, "h")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("i", range(len(plan.PRODUCTS)))
def test_products_backward(i, gated):
    m, n_in, n_out = (plan.PRODUCTS_GATED_BACKWARD if gated else plan.PRODUCTS)[i]
    dt, act = ("f16", "bf16")[(i + gated) % 2], ACTS[i % 4]
    assert plan.backward_route(m, n_out, n_in) == "product"
    print(f"backward product {m} {n_out} {n_in} {dt} {act} gated={gated}", flush=True)
    w, up = make_weight(n_out, n_in, 64, i + 100), make_weight(n_out, n_in, 64, i + 110)
    dy, pre, u = normal(12, (m, n_out), dt), normal(13, (m, n_out), dt, 2.0), normal(14, (m, n_out), dt)
    d64, p64, u64 = lc.to64(dy), lc.to64(pre), lc.to64(u)
    if gated:
        dx, dz, dup = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, dy, pre, u, activation=act)
        exact, _, bound = lc.slope_product_expected(dt, act, d64, p64, u64)
        lc.check(dz, exact, bound, "dgate")
        exact, bound = lc.value_product_expected(dt, act, d64, p64)
        lc.check(dup, exact, bound, "dup")
        left = np.concatenate([lc.to64(dz), lc.to64(dup)], 1)
        right = np.concatenate([lc.to64(weight_values(t, n_out, n_in, 64, dt)) for t in (w, up)])
    else:
        dx, dz, db = dq4.dq4_linear_fused_backward(**w, n_out=n_out, n_in=n_in, blocksize=64, dy=dy, pre=pre,
                                                   activation=act, bias_grad=True)
        exact, e, bound = lc.slope_product_expected(dt, act, d64, p64)
        lc.check(dz, exact, bound, "dz")
        gm = gamma_deterministic(m)
        lc.check(db, exact.sum(0), e.sum(0) * (1 + gm) + gm * np.abs(exact).sum(0) + 1e-37, "dbias")
        left, right = lc.to64(dz), lc.to64(weight_values(w, n_out, n_in, 64, dt))
    z, e = lc.product64(left, np.ascontiguousarray(right.T), dt)
    lc.check(dx, z, lc.rounding(dt, z, e), "dx")


# ----------------------------------------------------------------------------
# rows that do not mix, codes that no element uses
# ----------------------------------------------------------------------------
# (m, n_out, n_in, kernel forward linear, gated)
ISOLATION = [(2, 264, 2080, "token", "token"), (40, 264, 544, "batch", "batch"), (40, 264, 520, "ragged", "ragged"),
             (65, 28672, 544, "tile", "tile"), (129, 8200, 2048, "tile", "tile"), (100, 300, 6176, "tile", "tile"),
             (130, 201, 65, "product", "product")]


@pytest.mark.parametrize("m,n_out,n_in,linear,gated", ISOLATION)
def test_rows_do_not_mix(m, n_out, n_in, linear, gated):
    """Rows of NaN and infinities reach their own outputs only; the last row,
    beside the padding, is one of them."""
    assert plan.forward_route(m, n_out, n_in, False) == linear and plan.forward_route(m, n_out, n_in, True) == gated
    w, up = make_weight(n_out, n_in, 64, 120), make_weight(n_out, n_in, 64, 121)
    x, dy = normal(15, (m, n_in), "bf16"), normal(16, (m, n_out), "bf16")
    rows = [m - 1] if m < 4 else [1, m // 2, m - 1]
    others = [r for r in range(m) if r not in rows]

    def spoiled(t):
        bad = t.clone()
        bad[rows[0]] = float("nan")
        for r in rows[1:]:
            bad[r, -1] = float("inf")
        return bad
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)
    for name, call, t in (("linear", lambda v: dq4.dq4_linear_fused(**w, **sizes, x=v), x),
                          ("gated", lambda v: dq4.dq4_gated_fused(w, up, n_out, n_in, 64, v), x),
                          ("backward", lambda v: dq4.dq4_linear_fused_backward(**w, **sizes, dy=v)[0], dy)):
        a, b = call(t), call(spoiled(t))
        assert_bits_equal(bits_of(b[others].contiguous()), bits_of(a[others].contiguous()), name)
        assert bool(torch.isnan(b[rows[0]]).all()), name
        for r in rows[1:]:
            assert not bool(torch.isfinite(b[r]).all()), name


@pytest.mark.parametrize("m,n_out,n_in", [(65, 28672, 544), (65, 16400, 544), (129, 16400, 1056), (100, 300, 6176),
                                          (1, 70, 160), (40, 33, 544), (20, 33, 1000), (130, 201, 65), (130, 264, 520)])
def test_values_that_no_code_uses(m, n_out, n_in):
    """Infinities and NaN in codebook entries that no element names, code 0 and
    scale code 0 among them, which loads beyond a row or the weight give."""
    w = make_weight(n_out, n_in, 32, 122)
    packed = torch.where((w["packed"] & 15) == 0, w["packed"] | 1, w["packed"])
    packed = torch.where((packed >> 4) == 0, packed | 16, packed)
    plain = dict(w, packed=packed, scale_codes=torch.clamp(w["scale_codes"], min=1))
    bad = dict(plain, codebook4=w["codebook4"].clone(), scale_codebook=w["scale_codebook"].clone())
    bad["codebook4"][0], bad["scale_codebook"][0] = float("inf"), float("nan")
    x, dy = normal(17, (m, n_in), "bf16"), normal(18, (m, n_out), "bf16")
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=32)
    for name, call in (("linear", lambda t: dq4.dq4_linear_fused(**t, **sizes, x=x)),
                       ("gated", lambda t: dq4.dq4_gated_fused(t, t, n_out, n_in, 32, x)),
                       ("backward", lambda t: dq4.dq4_linear_fused_backward(**t, **sizes, dy=dy)[0]),
                       ("gated backward", lambda t: dq4.dq4_gated_fused_backward(t, t, n_out, n_in, 32, dy, dy, dy)[0])):
        a, b = call(plain), call(bad)
        assert bool(torch.isfinite(a).all()), name
        assert_bits_equal(bits_of(b), bits_of(a), name)


# ----------------------------------------------------------------------------
# every element of the weight, on every kernel that decodes
# ----------------------------------------------------------------------------
# (m, n_out, n_in, blocksize): one-hot rows read m columns (backward: m rows)
# of the weight a call
SELECT = [(1, 70, 160, 32), (2, 40, 2080, 64), (16, 47, 544, 32), (33, 50, 640, 64), (64, 70, 1056, 128),
          (3, 50, 2056, 32), (20, 90, 1000, 64), (37, 40, 168, 4096), (100, 300, 6176, 32), (65, 28672, 544, 64),
          (129, 8200, 2048, 64), (130, 201, 65, 32), (200, 512, 512, 64), (130, 264, 520, 64), (70, 33, 1001, 64),
          (5, 70001, 33, 64)]


def one_hot_calls(m, k):
    """(first index, rows) of the calls that select all of k."""
    for first in range(0, k, m):
        x = torch.zeros((m, k), device="cuda")
        rows = min(m, k - first)
        i = torch.arange(rows, device="cuda")
        x[i, first + i] = 1.0
        yield first, rows, x


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [-3.0, -12.0])
@pytest.mark.parametrize("m,n_out,n_in,bs", SELECT)
def test_every_weight_element(m, n_out, n_in, bs, scale, dt):
    """A row with a single 1 gives one column of W (backward: one row): sums of
    exact zeros and one value, so the very value that the dequantization writes
    (a zero may lose its sign).  With the small scale FP16 values are subnormal."""
    print(f"select {m} {n_out} {n_in} {bs} {dt} forward {plan.forward_route(m, n_out, n_in, False)} gated "
          f"{plan.forward_route(m, n_out, n_in, True)} backward {plan.backward_route(m, n_out, n_in)}", flush=True)
    offset = 0.03 if scale > -5 else 1e-6
    w, up = make_weight(n_out, n_in, bs, 130, scale, offset), make_weight(n_out, n_in, bs, 131, scale, offset)
    wv, uv = (weight_values(t, n_out, n_in, bs, dt) for t in (w, up))
    if scale < -5 and dt == "f16":
        assert bool(((wv != 0) & (wv.abs() < 2.0 ** -14)).float().mean() > 0.2)
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=bs)
    y, g, u = (torch.empty((n_in, n_out), dtype=T[dt], device="cuda") for _ in range(3))
    for first, rows, x in one_hot_calls(m, n_in):
        x = x.to(T[dt])
        y[first:first + rows] = dq4.dq4_linear_fused(**w, **sizes, x=x)[:rows]
        pre = torch.empty((2, m, n_out), dtype=T[dt], device="cuda")
        dq4.dq4_gated_fused(w, up, n_out, n_in, bs, x, gate_pre=pre[0], up_pre=pre[1])
        g[first:first + rows], u[first:first + rows] = pre[0][:rows], pre[1][:rows]
    assert torch.equal(y, wv.t()), "linear"
    assert torch.equal(g, wv.t()) and torch.equal(u, uv.t()), "gated"
    del y, g, u
    if n_out > 9000:
        return    # a call for every m of many rows
    dx, dg, du = (torch.empty((n_out, n_in), dtype=T[dt], device="cuda") for _ in range(3))
    for first, rows, x in one_hot_calls(m, n_out):
        x = x.to(T[dt])
        dx[first:first + rows] = dq4.dq4_linear_fused_backward(**w, **sizes, dy=x)[0][:rows]
        # relu at 1: dgate = dh up, dup = dh; silu at 0: dgate = dh up / 2, dup = 0
        zero, one = torch.zeros_like(x), torch.ones_like(x)
        du[first:first + rows] = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, bs, x, one, zero,
                                                              activation="relu")[0][:rows]
        dg[first:first + rows] = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, bs, x, zero, 2 * one,
                                                              activation="silu")[0][:rows]
    assert torch.equal(dx, wv), "backward"
    assert torch.equal(dg, wv) and torch.equal(du, uv), "gated backward"
