"""Float64 references and error bounds of the fused linear and gated calls.

No arithmetic of the dequantization lives here: weights come from the oracle,
as the values of the call's 16-bit type T.  The bounds are derived from the
arithmetic of the calls (include/dq4_linear.h):

* products of two T values are exact in FP32 (FP16: 22 significant bits, BF16:
  16); an FP32 sum of K of them in any order is within gamma_K S of the exact
  sum, S = sum |x| |w| (sum_bounds.gamma_deterministic);
* an FP32 addition or product adds at most u32 = 2^-24 of its result;
* an activation is evaluated in FP32 with a handful of operations on an
  exponential whose argument (at most z^2 / 2 + |z| + 2 in size, times log2 e)
  was rounded: a relative error of at most 4 u32 (z^2 + 16), and 4 u32 |z| where
  1 - tail cancels; below 2^-126 results may be flushed, which the subnormal
  term covers.  The erfc fit is within 1.2e-7 = 2.02 u32 of erfc;
* a bound L on |act'| carries the error of z into act(z);
* the one rounding to T adds u_T of the value (2^-11 FP16, 2^-8 BF16) and half
  the smallest subnormal.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from gpu_util import oracle_bits
from sum_bounds import U32, gamma_deterministic

TYPES = {"f16": (torch.float16, 2.0 ** -11, 2.0 ** -25),
         "bf16": (torch.bfloat16, 2.0 ** -8, 2.0 ** -134)}
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}
C = math.sqrt(2.0 / math.pi)


def to64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def weight64(x, dt: str) -> np.ndarray:
    bits = oracle_bits(x, dt)
    t = torch.from_numpy(bits.view(np.int16)).view(TYPES[dt][0])
    return t.to(torch.float64).numpy().reshape(x.n_rows, x.n_cols)


def _erfc(v):
    return torch.special.erfc(torch.from_numpy(v)).numpy()


def act64(name, z):
    with np.errstate(over="ignore"):
        if name == "none":
            return z
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "silu":
            return z / (1 + np.exp(-z))
        if name == "gelu":
            return 0.5 * z * _erfc(-z / math.sqrt(2))
        return z / (1 + np.exp(-2 * C * (z + 0.044715 * z ** 3)))


def slope64(name, z):
    with np.errstate(over="ignore"):
        if name == "none":
            return np.ones_like(z)
        if name == "relu":
            return (z > 0).astype(np.float64)
        if name == "silu":
            s = 1 / (1 + np.exp(-z))
            return s * (1 + z * (1 - s))
        if name == "gelu":
            return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        s = 1 / (1 + np.exp(-2 * C * (z + 0.044715 * z ** 3)))
        return s + z * s * (1 - s) * 2 * C * (1 + 3 * 0.044715 * z * z)


def act_error(name, z, value):
    """Bound on the FP32 evaluation of act at an exact z."""
    if name in ("none", "relu"):
        return np.zeros_like(z)
    return 4 * U32 * (np.abs(value) * (z * z + 16) + np.abs(z))


def slope_error(name, z):
    """Bound on the FP32 evaluation of act' at an exact z: its terms are s and
    z s (1 - s) v' (or z times the density), each at most 1 + z^2 in size and
    built from the exponential above."""
    if name in ("none", "relu"):
        return np.zeros_like(z)
    return 8 * U32 * (z * z + 16) * (1 + np.minimum(z * z, 16.0))


def rounding(dt, value, error):
    """error, plus the rounding of (value +- error) to T."""
    _, u, sub = TYPES[dt]
    return error + u * (np.abs(value) + error) + sub


def product64(x, w, dt):
    """x w^T and the bound on its FP32 evaluation."""
    return x @ w.T, gamma_deterministic(max(x.shape[1], 1)) * (np.abs(x) @ np.abs(w).T)


def check(got: torch.Tensor, exact: np.ndarray, bound: np.ndarray, what: str):
    g = to64(got)
    assert g.shape == exact.shape, (what, g.shape, exact.shape)
    err = np.abs(g - exact)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    print(f"{what}: worst err/bound {worst:.3f}", flush=True)
    assert np.isfinite(g).all(), what
    assert (err <= bound).all(), f"{what}: err/bound {worst:.3f} at {np.unravel_index(np.argmax(err / bound), err.shape)}"


def linear_expected(dt, act, x, w, bias=None, residual=None):
    """((z, bound of pre), (y, bound of y)) in float64."""
    z, e = product64(x, w, dt)
    if bias is not None:
        z = z + bias
        e = e + U32 * (np.abs(z) + e)
    a = act64(act, z)
    ea = LIPSCHITZ[act] * e + act_error(act, z, a)
    y = a
    if residual is not None:
        y = a + residual
        ea = ea + U32 * (np.abs(y) + ea)
    return (z, rounding(dt, z, e)), (y, rounding(dt, y, ea))


def gated_expected(dt, act, x, wg, wu):
    g, eg = product64(x, wg, dt)
    u, eu = product64(x, wu, dt)
    a = act64(act, g)
    ea = LIPSCHITZ[act] * eg + act_error(act, g, a)
    h = a * u
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu
    eh = eh + U32 * (np.abs(h) + eh)
    return (g, rounding(dt, g, eg)), (u, rounding(dt, u, eu)), (h, rounding(dt, h, eh))


def slope_product_expected(dt, act, dy, z, factor=None):
    """dy * factor * act'(z), the bound of its FP32 value and that of T's."""
    f = dy if factor is None else dy * factor
    s = slope64(act, z)
    exact = f * s
    e = np.abs(f) * slope_error(act, z) + 3 * U32 * np.abs(exact)
    return exact, e, rounding(dt, exact, e)


def value_product_expected(dt, act, dy, z):
    a = act64(act, z)
    exact = dy * a
    e = np.abs(dy) * act_error(act, z, a) + 2 * U32 * np.abs(exact)
    return exact, rounding(dt, exact, e)
