"""The fused calls where offsets pass 32 bits: weights of more than 2^32
elements, matrices of more than 2^31; and packed codes, scale codes and bias at
every alignment."""
from __future__ import annotations

import pytest

import block_wise_bit_amd as dq4

torch = pytest.importorskip("torch")

import linear_plan as plan  # noqa: E402
from gpu_util import assert_bits_equal, bits_of  # noqa: E402
from sum_bounds import gamma_deterministic  # noqa: E402
from test_linear_routes_gpu import T, make_weight, normal, weight_values  # noqa: E402

pytestmark = pytest.mark.gpu

HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("not enough free memory")
    from libs import ensure_hip_library
    ensure_hip_library()
    yield
    torch.cuda.empty_cache()


def close(got, a, b, dt, what):
    """got = T(a b^T) within the FP32 sum's bound and one rounding."""
    a, b = a.double(), b.double()
    exact, s = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    err, e = (got.double() - exact).abs(), gamma_deterministic(a.size(1)) * s
    bound = e + HALF[dt] * (exact.abs() + e) + 2.0 ** -25
    print(f"{what}: worst err/bound {float((err / bound).max()):.3f}", flush=True)
    assert bool((err <= bound).all()), what


# (m, n_out, n_in, forward, backward): 2^32 elements and more of weight
WEIGHTS = [(1, 1 << 21, 2080, "token", "columns"), (8, 1 << 21, 2080, "batch", "columns"),
           (20, 1 << 21, 2056, "ragged", "columns"), (130, 1 << 21, 2080, "tile", "product"),
           (130, 1 << 21, 2049, "product", "product"), (3, 2100, 1 << 21, "batch", "columns"),
           (66, 2100, 1 << 21, "tile", "columns"), (130, 2100, (1 << 21) - 1, "product", "product")]


@pytest.mark.parametrize("m,n_out,n_in,forward,backward", WEIGHTS)
def test_weights_of_more_than_2_to_32_elements(m, n_out, n_in, forward, backward):
    assert plan.forward_route(m, n_out, n_in, False) == forward and plan.backward_route(m, n_out, n_in) == backward
    dt = "bf16"
    print(f"far weight {m} {n_out} {n_in}", flush=True)
    w, up = make_weight(n_out, n_in, 64, 140), make_weight(n_out, n_in, 64, 141)
    x = normal(19, (m, n_in), dt)
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)
    rows = torch.cat([torch.arange(0, 70), torch.arange(n_out // 2 - 40, n_out // 2 + 40),
                      torch.arange(n_out - 70, n_out)]).cuda()

    def some_rows(t):
        return torch.cat([dq4.dq4_nested_dequant_rows(**t, n_rows=n_out, n_cols=n_in, r0=r0, rows=k, blocksize=64,
                                                      out_dtype=T[dt]).view(k, n_in)
                          for r0, k in ((0, 70), (n_out // 2 - 40, 80), (n_out - 70, 70))])
    y = dq4.dq4_linear_fused(**w, **sizes, x=x)
    close(y[:, rows], x, some_rows(w), dt, "linear")
    pre = torch.empty((2, m, n_out), dtype=T[dt], device="cuda")
    dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x, gate_pre=pre[0], up_pre=pre[1])
    close(pre[0][:, rows], x, some_rows(w), dt, "gate")
    close(pre[1][:, rows], x, some_rows(up), dt, "up")
    # gradients whose rows of dz are zero but where the weight's rows are known
    dy = torch.zeros((m, n_out), dtype=T[dt], device="cuda")
    dy[:, rows] = normal(20, (m, rows.numel()), dt)
    dx, _, _ = dq4.dq4_linear_fused_backward(**w, **sizes, dy=dy)
    part = dy[:, rows]
    keep = slice(None) if n_in < 10000 else torch.cat([torch.arange(0, 300), torch.arange(n_in - 300, n_in)]).cuda()
    close(dx[:, keep], part, some_rows(w)[:, keep].t().contiguous(), dt, "dx")
    one = torch.ones_like(dy)
    dx, _, _ = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, dy, one, one, activation="relu")
    both = torch.cat([some_rows(w), some_rows(up)])[:, keep]
    close(dx[:, keep], torch.cat([part, part], 1), both.t().contiguous(), dt, "gated dx")


@pytest.mark.parametrize("n_out,n_in", [(32768, 64), (32769, 65)])
def test_matrices_of_more_than_2_to_31_elements(n_out, n_in):
    m, dt = 70000, "bf16"
    print(f"far matrix {m} {n_out} {n_in}", flush=True)
    w, up = make_weight(n_out, n_in, 64, 150), make_weight(n_out, n_in, 64, 151)
    wv, uv = weight_values(w, n_out, n_in, 64, dt), weight_values(up, n_out, n_in, 64, dt)
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)
    x = normal(21, (m, n_in), dt)
    pre = torch.empty((m, n_out), dtype=T[dt], device="cuda")
    y = dq4.dq4_linear_fused(**w, **sizes, x=x, pre=pre)
    for rows in (slice(0, 200), slice(m // 2, m // 2 + 200), slice(m - 200, m)):
        close(y[rows], x[rows], wv, dt, "linear")
    assert torch.equal(y.view(torch.int16), pre.view(torch.int16))
    g, u = pre, torch.empty_like(pre)
    dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x, h=y, gate_pre=g, up_pre=u, activation="relu")
    for rows in (slice(0, 200), slice(m - 200, m)):
        close(g[rows], x[rows], wv, dt, "gate")
        close(u[rows], x[rows], uv, dt, "up")
    dy = y
    dy.fill_(0.0)
    dy[-300:] = normal(22, (300, n_out), dt)
    dx, _, db = dq4.dq4_linear_fused_backward(**w, **sizes, dy=dy, bias_grad=True)
    close(dx[-300:], dy[-300:], wv.t().contiguous(), dt, "dx")
    assert bool((dx[:-300] == 0).all())
    exact = dy[-300:].double().sum(0)
    assert bool(((db - exact).abs() <= gamma_deterministic(m) * dy[-300:].double().abs().sum(0)).all())
    one = g
    one.fill_(1.0)
    dx, dg, du = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, dy, one, one, activation="relu")
    assert torch.equal(dg.view(torch.int16), du.view(torch.int16))
    close(dx[-300:], torch.cat([dy[-300:], dy[-300:]], 1), torch.cat([wv, uv]).t().contiguous(), dt, "gated dx")
    assert bool((dx[:-300] == 0).all())


@pytest.mark.parametrize("skew", [1, 2, 3])
@pytest.mark.parametrize("m,n_out,n_in", [(1, 70, 96), (5, 33, 544), (70, 264, 520), (130, 201, 65), (200, 512, 512)])
def test_parts_of_a_weight_at_any_address(m, n_out, n_in, skew):
    """Packed codes 1 to 3 bytes off a dword (a kernel for it), scale codes and
    bias off any alignment (the aligned call's bits)."""
    w, up = make_weight(n_out, n_in, 64, 160), make_weight(n_out, n_in, 64, 161)

    def moved(t, by):
        big = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        big[by:] = t
        return big[by:]
    x, bias, dy = normal(23, (m, n_in), "f16"), normal(24, (n_out,), "f16"), normal(25, (m, n_out), "f16")
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)
    shifted = [dict(t, scale_codes=moved(t["scale_codes"], skew), nested_absmax=moved(t["nested_absmax"], skew),
                    codebook4=moved(t["codebook4"], skew), scale_codebook=moved(t["scale_codebook"], skew)) for t in (w, up)]

    def calls(a, b, bias):
        return (dq4.dq4_linear_fused(**a, **sizes, x=x, bias=bias), dq4.dq4_gated_fused(a, b, n_out, n_in, 64, x),
                dq4.dq4_linear_fused_backward(**a, **sizes, dy=dy)[0],
                dq4.dq4_gated_fused_backward(a, b, n_out, n_in, 64, dy, dy, dy)[0])
    for got, want in zip(calls(*shifted, moved(bias, skew)), calls(w, up, bias)):
        assert_bits_equal(bits_of(got), bits_of(want), "scales and bias at any address")
    off = [dict(t, packed=moved(t["packed"], skew)) for t in (w, up)]
    wv = weight_values(w, n_out, n_in, 64, "f16")
    close(dq4.dq4_linear_fused(**off[0], **sizes, x=x), x, wv, "f16", "linear")
    close(dq4.dq4_linear_fused_backward(**off[0], **sizes, dy=dy)[0], dy, wv.t().contiguous(), "f16", "dx")
    pre = torch.empty((2, m, n_out), dtype=torch.float16, device="cuda")
    dq4.dq4_gated_fused(*off, n_out, n_in, 64, x, gate_pre=pre[0], up_pre=pre[1])
    close(pre[0], x, wv, "f16", "gate")
    close(pre[1], x, weight_values(up, n_out, n_in, 64, "f16"), "f16", "up")


@pytest.mark.parametrize("m,n_out,n_in", [(2, 264, 512), (20, 264, 520), (40, 264, 544), (65, 100, 8192), (300, 264, 512),
                                          (300, 201, 65)])
def test_row_strides_above_2_to_22(m, n_out, n_in):
    """Rows 2^22 + 8 elements apart: the dense call's bits."""
    ld = (1 << 22) + 8
    w, up = make_weight(n_out, n_in, 64, 170), make_weight(n_out, n_in, 64, 171)
    sizes = dict(n_out=n_out, n_in=n_in, blocksize=64)

    def far(t):
        view = torch.empty((t.size(0) - 1) * ld + t.size(1), dtype=t.dtype, device="cuda").as_strided(t.shape, (ld, 1))
        view.copy_(t)
        return view
    x, res, pre = normal(26, (m, n_in), "bf16"), normal(27, (m, n_out), "bf16"), normal(28, (m, n_out), "bf16")
    y = far(torch.zeros_like(res))
    dq4.dq4_linear_fused(**w, **sizes, x=far(x), residual=far(res), y=y)
    assert_bits_equal(bits_of(y.contiguous()), bits_of(dq4.dq4_linear_fused(**w, **sizes, x=x, residual=res)), "linear")
    h = dq4.dq4_gated_fused(w, up, n_out, n_in, 64, far(x))
    assert_bits_equal(bits_of(h), bits_of(dq4.dq4_gated_fused(w, up, n_out, n_in, 64, x)), "gated")
    kw = dict(activation="gelu", bias_grad=True)
    got = dq4.dq4_linear_fused_backward(**w, **sizes, dy=far(res), pre=far(pre), dx=far(torch.zeros_like(x)),
                                        dz=far(torch.zeros_like(res)), **kw)
    for a, b in zip(got, dq4.dq4_linear_fused_backward(**w, **sizes, dy=res, pre=pre, **kw)):
        assert_bits_equal(bits_of(a.contiguous()), bits_of(b), "linear backward")
    got = dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, far(res), far(pre), far(pre), dgate=far(torch.zeros_like(res)),
                                       dup=far(torch.zeros_like(res)))
    for a, b in zip(got, dq4.dq4_gated_fused_backward(w, up, n_out, n_in, 64, res, pre, pre)):
        assert_bits_equal(bits_of(a.contiguous()), bits_of(b), "gated backward")
