"""Test oracle of the routed-expert operators: plain NumPy in fp64.

Test infrastructure only; the product path never imports it. Definitions as
in include/lora_mi355x.h, with explicit loops where the method has choices.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def route(logits, top_k, scores="softmax", bias=None, groups=1, top_groups=None,
          group_score="max", renormalize=True, scaling=1.0):
    """(ids int32 [T, k], weights fp64 [T, k], choice fp64 [T, E]) of logits [T, E].

    `choice` is each expert's score with its bias, -inf where the expert is
    not available, before any group drops out."""
    x = np.asarray(logits, np.float64).copy()
    T, E = x.shape
    shut = np.isnan(x) | (x == -np.inf)
    x = np.minimum(x, float(np.finfo(np.float32).max))
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    choice = np.full((T, E), -np.inf)
    top_groups = groups if top_groups is None else top_groups
    for t in range(T):
        open_ = ~shut[t]
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if scores == "softmax":
                if open_.any():
                    e = np.exp(x[t, open_] - x[t, open_].max())
                    s[open_] = e / e.sum()
            else:
                s[open_] = 1.0 / (1.0 + np.exp(-x[t, open_]))
        c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        c[shut[t] | np.isnan(c)] = -np.inf
        choice[t] = c
        live = c.copy()
        if top_groups < groups:
            per = E // groups
            worth = []
            for g in range(groups):
                best = sorted((v for v in c[g * per:(g + 1) * per] if v != -np.inf), reverse=True)
                best = best[:2 if group_score == "sum2" else 1]
                worth.append(sum(best) if best else -np.inf)
            order = sorted(range(groups), key=lambda g: (-worth[g], g))
            for g in order[top_groups:]:
                live[g * per:(g + 1) * per] = -np.inf
        order = sorted(range(E), key=lambda e: (-live[e], e))[:top_k]
        for j, e in enumerate(order):
            if live[e] != -np.inf:
                ids[t, j] = e
                weights[t, j] = s[e]
        total = weights[t].sum()
        if renormalize:
            weights[t] = weights[t] / total if total > 0 else 0.0
        weights[t] *= scaling
    return ids, weights, choice


def expert_rows(ids, num_experts, token_slot=None):
    """(row_token, positions, offsets, row_slot) of the choices ids [T, k]."""
    ids = np.asarray(ids)
    T, k = ids.shape
    flat = [(int(e) if 0 <= e < num_experts else num_experts, i)
            for i, e in enumerate(ids.reshape(-1))]
    order = sorted(flat)
    row_token = np.array([i // k for _, i in order], np.int32).reshape(-1)
    positions = np.full(T * k, -1, np.int32)
    offsets = np.zeros(num_experts + 1, np.int32)
    row_slot = np.full(T * k, -1, np.int32)
    for r, (e, i) in enumerate(order):
        if e < num_experts:
            positions[i] = r
            offsets[e + 1:] += 1
            if token_slot is not None:
                row_slot[r] = token_slot[i // k]
    return row_token, positions.reshape(T, k), offsets, row_slot


def quantize(x):
    """MXFP4 of x [rows, K]: (codes uint8 [rows, K / 2], scales uint8 [rows, ld])."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(2)
    _, e = np.frexp(top)   # top = m 2^e, m in [0.5, 1): floor(log2(top)) = e - 1
    byte = np.where(top > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0).astype(np.int64)
    a = np.abs(b) / np.exp2(byte - 127.0)[:, :, None]
    code = np.zeros(a.shape, np.int64)
    for i in range(1, 8):   # past the midpoint, or on it where the upper code is even
        mid = (GRID[i - 1] + GRID[i]) / 2
        code = np.where((a > mid) | ((a == mid) & (i % 2 == 0)), i, code)
    code += 8 * np.signbit(b)
    code = np.where(bad[:, :, None], 0, code).reshape(rows, K)
    scales = np.zeros((rows, -(-(K // 32) // 4) * 4), np.uint8)
    scales[:, :K // 32] = np.where(bad, 255, byte)
    return (code[:, 0::2] + 16 * code[:, 1::2]).astype(np.uint8), scales


def dequantize(codes, scales):
    """The fp64 values of MXFP4 rows."""
    codes = np.asarray(codes)
    rows, half = codes.shape
    c = np.stack([codes & 15, codes >> 4], 2).reshape(rows, half * 2)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = np.asarray(scales)[:, :half * 2 // 32].astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return v * np.repeat(s, 32, 1)


def expert_linear(x, w, offsets):
    """y [rows, N]: row r of expert e times w[e]^T; rows of no expert 0 (values)."""
    y = np.zeros((x.shape[0], w[0].shape[0]))
    for e in range(len(w)):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = x[lo:hi] @ w[e].T
    return y


def combine(rows, positions, weights, residual=None):
    """y[t] = residual[t] + sum over j of weights[t, j] rows[positions[t, j]]."""
    rows = np.asarray(rows, np.float64)
    T, k = positions.shape
    y = np.zeros((T, rows.shape[1])) if residual is None else np.asarray(residual, np.float64).copy()
    for t in range(T):
        for j in range(k):
            p = int(positions[t, j])
            if 0 <= p < rows.shape[0]:
                y[t] += float(weights[t, j]) * rows[p]
    return y
