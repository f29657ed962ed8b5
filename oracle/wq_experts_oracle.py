"""CPU oracle of the expert operators: routing, lists by expert, the experts' 4-bit products.

Everything in float64, one token and one pair at a time, from the operators' definitions as
``include/wq.h`` states them; the prepacked expert layout is restated plainly, so that the CUDA
layout pass can be compared with it byte for byte.
"""
from __future__ import annotations

import math

import numpy as np

from .wq_oracle import NIBBLE_POS_W4A16, TILE_K, dequant, unpack_codes

__all__ = ["route_experts", "expert_lists", "experts_product", "experts_gated", "experts_combine",
           "prepacked_bytes_experts", "prepack_experts", "EXPERT_UNIT_N"]

EXPERT_UNIT_N = 32


def _descending(values, allowed):
    """Indices of the allowed values, largest first, ties by the lower index."""
    return sorted((i for i in range(len(values)) if allowed[i]), key=lambda i: (-values[i], i))


def route_experts(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True,
                  scale=1.0):
    """(idx int32 [T, top_k], w float64 [T, top_k]); -1 and 0 where no expert is left."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    idx = np.full((T, top_k), -1, dtype=np.int32)
    w = np.zeros((T, top_k))
    size = E // groups
    for t in range(T):
        x = [float(v) for v in logits[t]]
        finite = [math.isfinite(v) for v in x]
        p = [0.0] * E
        if score == "softmax":
            top = max([v for v, f in zip(x, finite) if f], default=0.0)
            e = [math.exp(v - top) if f else 0.0 for v, f in zip(x, finite)]
            total = math.fsum(e)
            if total > 0:
                p = [v / total for v in e]
        else:
            for i in range(E):
                if finite[i]:
                    p[i] = 1.0 / (1.0 + math.exp(-x[i])) if x[i] > -700 else math.exp(x[i])
        b = [0.0] * E if bias is None else [float(v) for v in bias]
        allowed = [f and math.isfinite(v) for f, v in zip(finite, b)]
        c = [pi + bi for pi, bi in zip(p, b)]
        if top_groups < groups:
            value, has = [], []
            for j in range(groups):
                members = _descending(c[j * size:(j + 1) * size], allowed[j * size:(j + 1) * size])[:group_top]
                has.append(bool(members))
                value.append(sum(c[j * size + m] for m in members) if members else 0.0)
            stay = set(_descending(value, has)[:top_groups])
            allowed = [a and i // size in stay for i, a in enumerate(allowed)]
        chosen = _descending(x if bias is None else c, allowed)[:top_k]
        total = math.fsum(p[i] for i in chosen)
        for j, i in enumerate(chosen):
            idx[t, j] = i
            w[t, j] = (p[i] if not renorm else p[i] / total if total > 0 else 0.0) * scale
    return idx, w


def expert_lists(idx, E):
    """(offsets int32 [E + 1], rows: the listed pairs only)."""
    flat = np.asarray(idx).reshape(-1)
    rows, offsets = [], [0]
    for e in range(E):
        rows += [p for p in range(flat.size) if flat[p] == e]
        offsets.append(len(rows))
    return np.array(offsets, dtype=np.int32), np.array(rows, dtype=np.int32)


def experts_product(A, Q, s, g, idx, by_pair=False):
    """(y, absdot), float64 [T * top_k, N]: A[p // top_k] (or A[p]) . W_idx[p]; NaN where idx is no expert."""
    flat = np.asarray(idx).reshape(-1)
    top_k = np.asarray(idx).shape[1]
    A = np.asarray(A).astype(np.float64)
    E, N = Q.shape[0], Q.shape[2]
    y = np.full((flat.size, N), np.nan)
    ad = np.full((flat.size, N), np.nan)
    for e in range(E):
        pairs = np.flatnonzero(flat == e)
        if pairs.size:
            W = dequant(unpack_codes(Q[e]), s[e], g)
            a = A[pairs if by_pair else pairs // top_k]
            y[pairs] = a @ W
            ad[pairs] = np.abs(a) @ np.abs(W)
    return y, ad


def experts_gated(y):
    """silu(gate) * up of the columns [gate | up]."""
    half = y.shape[1] // 2
    gate, up = y[:, :half], y[:, half:]
    return gate / (1.0 + np.exp(-gate)) * up


def experts_combine(y, idx, w):
    """sum over j of w[t, j] * y[t * top_k + j]; choices that are no expert (NaN rows) add nothing."""
    T, top_k = np.asarray(idx).shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(top_k):
            if not np.isnan(y[t * top_k + j]).all():
                out[t] += np.float64(w[t, j]) * y[t * top_k + j]
    return out


def _units(N):
    return -(-N // EXPERT_UNIT_N)


def prepacked_bytes_experts(E, K, N, g):
    one = _units(N) * (K // TILE_K) * 2048 + _units(N) * (K // g) * 64
    return E * (-(-one // 128) * 128)


def prepack_experts(Q, s, g, gated=False):
    """The prepacked buffer (uint8), padding bytes between experts zero.

    Word ``((rt*2 + h)*32 + 4*gc + q)*4 + c`` of unit (u, kb) holds column ``32u + 16rt + 8h + gc``,
    rows ``128kb + 32c + 8i + 2q + b``, code 2i + b at nibble NIBBLE_POS_W4A16[2i + b]; then the scales."""
    E, K8, N = Q.shape
    K = K8 * 8
    stride = prepacked_bytes_experts(1, K, N, g)
    out = np.zeros(E * stride, dtype=np.uint8)
    NU, KT, G = _units(N), K // TILE_K, K // g
    for e in range(E):
        q = unpack_codes(Q[e])
        full = np.full((K, NU * 32), 8, dtype=np.uint32)
        sc = np.zeros((G, NU * 32), dtype=np.float16)
        for v in range(N):
            n = v if not gated else (v // 16) * 8 + v % 8 + (N // 2 if v & 8 else 0)
            full[:, v] = q[:, n]
            sc[:, v] = s[e][:, n]
        words = np.zeros((NU, KT, 512), dtype=np.uint32)
        for col in range(32):
            for c in range(4):
                for qq in range(4):
                    at = ((col // 8) * 32 + 4 * (col % 8) + qq) * 4 + c
                    for j in range(8):
                        v = full[32 * c + 8 * (j // 2) + 2 * qq + j % 2::TILE_K, col::32]  # [KT, NU]
                        words[:, :, at] |= v.T << np.uint32(4 * NIBBLE_POS_W4A16[j])
        scales = np.zeros((NU, G, 32), dtype=np.float16)
        for col in range(32):
            scales[:, :, 4 * (col % 8) + 2 * (col // 16) + (col // 8) % 2] = sc[:, col::32].T
        body = np.concatenate([words.reshape(-1).view(np.uint8), scales.reshape(-1).view(np.uint8)])
        out[e * stride:e * stride + body.size] = body
    return out
