"""NaN and infinities in the saved pre-activations of the fused calls' backward
passes (include/dq4_linear.h): a NaN reaches every gradient that the formula
takes it to, whatever the activation; at the infinities, which a saved FP16
pre-activation reaches by overflow, act and act' take their limits."""
from __future__ import annotations

import numpy as np
import pytest

import block_wise_bit_amd as dq4
from block_wise_bit_amd import inputs

torch = pytest.importorskip("torch")

import linear_cases as lc  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
NAN, INF = float("nan"), float("inf")
# few rows (gradients decoded in registers), the product, slopes of one column
# a thread (odd width)
SIZES = [(3, 264, 128), (150, 264, 128), (150, 201, 65)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


def make_weight(n_out, n_in, seed):
    x = inputs.make_inputs(n_out * n_in, 64, "nf4", 0.03, seed=seed, n_rows=n_out, n_cols=n_in)
    return dict(dq4.to_device(x), offset=float(x.offset))


def normal(rng, shape, dt):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(lc.TYPES[dt][0]).cuda()


def planted(rng, m, n, dt):
    """A pre-activation with a NaN at [1, 5] and infinities at [0, 3], [0, 4]."""
    t = normal(rng, (m, n), dt)
    t[1, 5], t[0, 3], t[0, 4] = NAN, INF, -INF
    return t


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n_out,n_in", SIZES)
def test_linear_backward(m, n_out, n_in, act, dt):
    print(f"linear backward {m} {n_out} {n_in} {act} {dt}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m))
    w = make_weight(n_out, n_in, 3)
    dy, pre = normal(rng, (m, n_out), dt), planted(rng, m, n_out, dt)
    kw = dict(n_out=n_out, n_in=n_in, blocksize=64, dy=dy, activation=act, bias_grad=True)
    dx, dz, db = dq4.dq4_linear_fused_backward(**w, **kw, pre=pre)
    assert bool(torch.isnan(dz[1, 5]))
    assert bool(torch.isnan(dx[1]).all()) and bool(torch.isnan(db[5]))
    assert float(dz[0, 3]) == float(dy[0, 3]) and float(dz[0, 4]) == 0.0
    # nothing else is reached
    finite = pre.clone()
    finite[1, 5], finite[0, 3], finite[0, 4] = 0.0, 0.0, 0.0
    dx0, dz0, db0 = dq4.dq4_linear_fused_backward(**w, **kw, pre=finite)
    keep = torch.ones_like(dz, dtype=torch.bool)
    keep[1, 5] = keep[0, 3] = keep[0, 4] = False
    assert torch.equal(dz[keep], dz0[keep])
    assert torch.equal(dx[2:], dx0[2:]) and bool(torch.isfinite(dx[0]).all())
    cols = [c for c in range(n_out) if c not in (3, 4, 5)]
    assert torch.equal(db[cols], db0[cols])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n_ff,n_in", SIZES)
def test_gated_backward(m, n_ff, n_in, act, dt):
    print(f"gated backward {m} {n_ff} {n_in} {act} {dt}", flush=True)
    rng = np.random.Generator(np.random.PCG64(m + 1))
    gate, up = make_weight(n_ff, n_in, 4), make_weight(n_ff, n_in, 5)
    dh, u, g = normal(rng, (m, n_ff), dt), normal(rng, (m, n_ff), dt), planted(rng, m, n_ff, dt)
    dx, dgate, dup = dq4.dq4_gated_fused_backward(gate, up, n_ff, n_in, 64, dh, g, u, activation=act)
    assert bool(torch.isnan(dgate[1, 5])) and bool(torch.isnan(dup[1, 5]))
    assert bool(torch.isnan(dx[1]).all())
    product = (dh[0, 3].float() * u[0, 3].float()).to(dh.dtype)
    assert float(dgate[0, 3]) == float(product) and float(dgate[0, 4]) == 0.0
    assert float(dup[0, 3]) == float(dh[0, 3].float() * INF) and float(dup[0, 4]) == 0.0
    finite = g.clone()
    finite[1, 5], finite[0, 3], finite[0, 4] = 0.0, 0.0, 0.0
    dx0, dgate0, dup0 = dq4.dq4_gated_fused_backward(gate, up, n_ff, n_in, 64, dh, finite, u, activation=act)
    keep = torch.ones_like(dgate, dtype=torch.bool)
    keep[1, 5] = keep[0, 3] = keep[0, 4] = False
    assert torch.equal(dgate[keep], dgate0[keep]) and torch.equal(dup[keep], dup0[keep])
    assert torch.equal(dx[2:], dx0[2:])


@pytest.mark.parametrize("act", ["none"] + ACTS)
@pytest.mark.parametrize("m,n_out,n_in", [(1, 264, 128), (9, 264, 128), (150, 264, 128), (150, 201, 65)])
def test_forward_keeps_nan(m, n_out, n_in, act):
    """A NaN in one column of bias reaches that column of every row, no other."""
    rng = np.random.Generator(np.random.PCG64(m + 2))
    w = make_weight(n_out, n_in, 6)
    x, bias = normal(rng, (m, n_in), "bf16"), normal(rng, (n_out,), "bf16")
    bad = bias.clone()
    bad[7] = NAN
    kw = dict(n_out=n_out, n_in=n_in, blocksize=64, x=x, activation=act)
    pre = torch.empty((m, n_out), dtype=x.dtype, device="cuda")
    y, y0 = dq4.dq4_linear_fused(**w, **kw, bias=bad, pre=pre), dq4.dq4_linear_fused(**w, **kw, bias=bias)
    assert bool(torch.isnan(y[:, 7]).all()) and bool(torch.isnan(pre[:, 7]).all())
    cols = [c for c in range(n_out) if c != 7]
    assert torch.equal(y[:, cols], y0[:, cols])
