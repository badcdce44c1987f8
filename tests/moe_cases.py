"""Inputs, 64-bit references and error bounds of the mixture-of-experts layer
(include/dq4_moe.h).  The bounds count the roundings of the calls, as
linear_cases.py does for the linear and gated ones:

* logits: products of two T values are exact in FP32, their sums run in FP64; the
  choice is compared exactly on inputs whose sums are exact in FP64;
* weights: the exponent's rounding and exp2's and the reciprocal's last place, and
  a sum of up to 512 terms, each at most |l - top| 2^-22 + 2^-21 relative.  The
  exponential instruction gives 0 for results below 2^-126, the smallest normal
  number, and the sum they are divided by is at least 1 (the largest logit's own
  term): 2^-126 absolute, and again 2^-126 for the product with the reciprocal;
* h: the gated call's bound, rounded to T;
* y: an FP32 sum of n_ff products of two T values per expert, the product with
  the weight and the sum over the experts (8 partial sums, top_k experts), the
  residual, and the rounding to T.  h's own error passes through |Wd|.
"""
from __future__ import annotations

import numpy as np
import torch

from block_wise_bit_amd import inputs
from linear_cases import TYPES, check, gated_expected, rounding, to64, weight64  # noqa: F401
from sum_bounds import U32, gamma_deterministic


class Layer:
    """Stacked weights of random experts, on the host."""

    def __init__(self, n_experts, n_ff, n_in, blocksize, seed=0):
        self.sizes = (n_experts, n_ff, n_in)
        self.blocksize = blocksize
        make = lambda rows, cols, i: inputs.make_inputs(  # noqa: E731
            rows * cols, blocksize, ("nf4", "fp4", "nf4")[i], (0.03, -0.02, 0.01)[i],
            seed=inputs.SEED_BASE + 1000 + 3 * seed + i, n_rows=rows, n_cols=cols)
        self.host = [make(n_experts * n_ff, n_in, 0), make(n_experts * n_ff, n_in, 1),
                     make(n_experts * n_in, n_ff, 2)]

    def device(self):
        import block_wise_bit_amd as dq4
        return [dict(dq4.to_device(h), offset=float(h.offset)) for h in self.host]

    def matrices(self, dt):
        E, n_ff, n_in = self.sizes
        g, u, d = (weight64(h, dt) for h in self.host)
        return g.reshape(E, n_ff, n_in), u.reshape(E, n_ff, n_in), d.reshape(E, n_in, n_ff)


def moe64(dt, act, layer, x, ids, weights, residual=None):
    """(y, bound) in float64; x, residual: T tensors; ids, weights: arrays."""
    E, n_ff, n_in = layer.sizes
    wg, wu, wd = layer.matrices(dt)
    xv = to64(x)
    m, k = ids.shape
    y, e, mag = np.zeros((m, n_in)), np.zeros((m, n_in)), np.zeros((m, n_in))
    for ex in range(E):
        share = np.where(ids == ex, weights.astype(np.float64), 0.0).sum(axis=1)
        rows = np.flatnonzero((ids == ex).any(axis=1))
        if rows.size == 0:
            continue
        _, _, (h, eh) = gated_expected(dt, act, xv[rows], wg[ex], wu[ex])
        w = share[rows, None]
        out = h @ wd[ex].T
        size = np.abs(w) * ((np.abs(h) + eh) @ np.abs(wd[ex]).T)
        y[rows] += w * out
        e[rows] += np.abs(w) * (eh @ np.abs(wd[ex]).T)
        mag[rows] += size * (1 + k * U32)  # (weights of an expert that occurs twice are added up)
    e += gamma_deterministic(n_ff + k + 12) * mag + k * U32 * mag
    if residual is not None:
        r = to64(residual)
        y = y + r
        e = e + U32 * (np.abs(y) + e)
    return y, rounding(dt, y, e)


def route64(x, router, top_k, bias=None, renormalize=True):
    logits = to64(x) @ to64(router).T
    if bias is not None:
        logits = logits + bias.astype(np.float64)
    m, E = logits.shape
    ids, weights = np.full((m, top_k), -1), np.zeros((m, top_k))
    bound = np.zeros((m, top_k))
    for t in range(m):
        l = logits[t]
        order = sorted(range(E), key=lambda e: (np.isnan(l[e]), -l[e] if not np.isnan(l[e]) else 0.0, e))
        order = [e for e in order if l[e] != -np.inf][:top_k]
        ids[t, :len(order)] = order
        with np.errstate(invalid="ignore"):
            top = l[order[0]] if order else 0.0
            p = np.exp(l - top)
        total = p[order].sum() if renormalize else p.sum()
        if order:
            weights[t, :len(order)] = np.nan if np.isnan(l).any() else p[order] / total
        with np.errstate(invalid="ignore"):
            reach = np.abs(np.where(np.isfinite(l), l - top, 0.0)).max(initial=0.0)
        bound[t] = (reach * 2.0 ** -21 + 2.0 ** -19) * np.abs(weights[t]) + 2.0 ** -125
    return ids, weights, bound
