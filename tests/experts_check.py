"""Inputs and error bounds of the expert operators' tests (shared by the CPU and the GPU file).

Bounds, derived before any run. A product sums K exact products of fp16 values in K/16 matrix
instructions and at most 16 further fp32 additions, each off by at most 2^-22 of the sum of
magnitudes S = sum |a w| (the instruction may truncate its 16 + 1 addends):
    sum:   |d - d*| <= (K/16 + 16) 2^-22 S, plus 2^-23 |d| for the fp32 scale product
    fp16:  half a step, 2^-11 |y|, or 2^-25 where y is below the normal range.
Gated: silu' lies in [-0.1, 1.1], so the errors of the sums enter as 1.1 |up| eg + |silu| eu,
and fp32 exp, division and products add less than 2^-18 |h| (exp's error grows with |gate| <= 40).
Combine: every pair's product is rounded once to fp16 before the weighted sum, which is fp32.
"""
from __future__ import annotations

import math

import numpy as np

import oracle


def half_step(y):
    return np.maximum(2.0 ** -11 * np.abs(y), 2.0 ** -25)


def sum_bound(y, absdot, K):
    return (K / 16 + 16) * 2.0 ** -22 * absdot + 2.0 ** -23 * np.abs(y)


def product_bound(y, absdot, K):
    e = sum_bound(y, absdot, K)
    return e + half_step(np.abs(y) + e)


def gated_bound(y, absdot, K):
    e = sum_bound(y, absdot, K)
    half = y.shape[1] // 2
    gate, up = y[:, :half], y[:, half:]
    silu = gate / (1.0 + np.exp(-gate))
    eh = 1.1 * (np.abs(up) + e[:, half:]) * e[:, :half] + np.abs(silu) * e[:, half:]
    h = silu * up
    eh = eh + 2.0 ** -18 * np.abs(h)
    return eh + half_step(np.abs(h) + eh)


def combine_bound(y, absdot, idx, w, K):
    T, top_k = idx.shape
    e = product_bound(y, absdot, K)
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for j in range(top_k):
            p = t * top_k + j
            if not np.isnan(y[p]).all():
                out[t] += abs(float(w[t, j])) * e[p]
                mag[t] += abs(float(w[t, j])) * (np.abs(y[p]) + e[p])
    out = out + 2.0 ** -23 * (top_k + 1) * mag
    return out + half_step(mag)


def experts_inputs(E, K, N, g, T, top_k, seed=0, padded=0.0, by_pair=False, skew=0.0):
    rng = np.random.default_rng(seed)
    Q = rng.integers(0, 1 << 32, (E, K // 8, N), dtype=np.uint32).view(np.int32)
    s = ((0.5 + rng.random((E, K // g, N))) * 0.22 / math.sqrt(K)).astype(np.float16)
    A = rng.standard_normal((T * top_k if by_pair else T, K)).astype(np.float16)
    like = rng.standard_normal(E) * skew
    idx = np.argsort(-(like + rng.gumbel(size=(T, E))), axis=1)[:, :top_k].astype(np.int32)
    if padded:
        idx[rng.random(T) < padded] = -1
    w = (0.05 + rng.random((T, top_k))).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    offsets, rows = oracle.expert_lists(idx, E)
    rows = np.concatenate([rows, np.full(T * top_k - rows.size, -12345, dtype=np.int32)]).astype(np.int32)
    return {"Q": Q, "s": s, "A": A, "idx": idx, "w": w, "offsets": offsets, "rows": rows}


def combine_bound_once(y, absdot, idx, w, K):
    """The weighted sum with one rounding, the output's: the pairs' products enter as fp32 sums.

    A pair's sum as in sum_bound, its scale times w one rounding more (2^-24). The sum over the choices:
    top_k products and additions of 2^-24 of the magnitudes each; where the choices' k-blocks are added to
    one running sum, at most K/32 additions a choice (a scale per 32 rows) of 2^-24 of all that is
    in the sum, for top_k choices."""
    T, top_k = idx.shape
    err, mag, out = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(top_k):
            p = t * top_k + j
            if not np.isnan(y[p]).all():
                out[t] += float(w[t, j]) * y[p]
                err[t] += abs(float(w[t, j])) * (sum_bound(y[p], absdot[p], K) + 2.0 ** -24 * absdot[p])
                mag[t] += abs(float(w[t, j])) * absdot[p]
    err = err + 2.0 ** -24 * (2 * top_k + top_k * K / 32) * mag
    return err + half_step(np.abs(out) + err)
