"""Inputs, 64-bit references and error bounds of the LLM.int8 linear layer
(include/dq4_int8.h).  The bounds count the roundings of the calls:

* codes, scales and outlier lists are exact: 127 x / s is a quotient of short
  integers, so its FP64 value lies on a half only if it is one;
* the integer sum is exact; its FP32 value, the constant 1/127^2, and the three
  products with it and with the two scales are five roundings of u32 = 2^-24;
* products of two T values are exact in FP32, and an FP32 sum of L of them and
  what it is added to is within gamma_{L + 1} of the sum of magnitudes
  (sum_bounds.gamma_deterministic); bias and residual add one rounding each;
* the rounding to T adds u_T of the value and half the smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

from linear_cases import TYPES, check, rounding, to64  # noqa: F401  (re-exported)
from sum_bounds import U32, gamma_deterministic

R127 = np.float32(1.0) / np.float32(127.0)
assert R127.view(np.uint32) == 0x3C010204


def tokens(rng, m, k, dt, outliers=0, scale=1.0):
    """A normal bulk below 5.5 and some columns above the threshold of 6."""
    x = np.clip(rng.standard_normal((m, k)), -5.5, 5.5) * scale
    cols = np.sort(rng.choice(k, size=min(outliers, k), replace=False)) if outliers else np.zeros(0, np.int64)
    if m:
        x[:, cols] = x[:, cols] * 4 + np.where(x[:, cols] < 0, -8.0, 8.0)
    return torch.from_numpy(x).to(TYPES[dt][0])


def quant64(x: torch.Tensor, threshold: float):
    """(codes, scales, outliers or None) of the definition."""
    v = to64(x)
    m, k = v.shape
    with np.errstate(invalid="ignore"):
        big = ~(np.abs(v) < threshold) if threshold > 0 else np.zeros_like(v, bool)
    scales = np.max(np.where(big, 0.0, np.abs(v)), axis=1, initial=0.0)
    codes = np.zeros((m, k), np.int64)
    for i in range(m):
        if scales[i] > 0 and np.isfinite(scales[i]):
            codes[i] = np.where(big[i], 0, np.rint(127.0 * np.where(big[i], 0.0, v[i]) / scales[i]))
    scales = np.where(np.isfinite(scales), scales, np.nan)
    if threshold == 0:
        return codes, scales, None
    cols = np.flatnonzero(big.any(axis=0))
    codes[:, cols] = 0
    listed = np.full(1 + k, -1, np.int64)
    listed[0] = cols.size
    listed[1:1 + cols.size] = cols
    return codes, scales, listed


def weight(rng, n, k):
    return (torch.from_numpy(rng.integers(-128, 128, (n, k), dtype=np.int8)),
            torch.from_numpy((rng.random(n) * 0.08 + 0.02).astype(np.float32)))


def weight64(CB: torch.Tensor, SCB: torch.Tensor, dt: str) -> np.ndarray:
    """The 16-bit weight, with the rounding order of dq4_int8_prep."""
    v = (CB.cpu().numpy().astype(np.float32) * SCB.cpu().numpy()[:, None]) * R127
    return to64(torch.from_numpy(v).to(TYPES[dt][0]))


def linear64(dt, codes, scales, CB, SCB, bias=None, residual=None, x=None, cols=()):
    """(y, bound) in float64; arrays of values."""
    c, w = np.asarray(codes, np.float64), CB.cpu().numpy().astype(np.float64)
    z = (c @ w.T) * np.asarray(scales, np.float64)[:, None] * SCB.cpu().numpy().astype(np.float64) / 16129.0
    e = 5.01 * U32 * np.abs(z)
    if len(cols):
        w16 = weight64(CB, SCB, dt)[:, cols]
        xo = to64(x)[:, cols]
        mag = np.abs(z) + np.abs(xo) @ np.abs(w16).T
        z = z + xo @ w16.T
        e = e + gamma_deterministic(len(cols) + 33) * (mag + e)  # whole chunks of 32, with zeros
    for add in (bias, residual):
        if add is not None:
            z = z + add
            e = e + U32 * (np.abs(z) + e)
    return z, rounding(dt, z, e)


def backward64(dt, dy, CB, SCB):
    w = weight64(CB, SCB, dt)
    g = to64(dy)
    dx = g @ w
    e = gamma_deterministic(max(g.shape[1], 1)) * (np.abs(g) @ np.abs(w))
    db = g.sum(axis=0)
    eb = gamma_deterministic(max(g.shape[0], 1)) * np.abs(g).sum(axis=0)
    return (dx, rounding(dt, dx, e)), (db, eb + 1e-300)
