"""Plain CPU forms (numpy, fp64) of the operators on rows grouped by a device-side id:
the stable sort of token-expert pairs, dispatch, combination with weights, its
gradient, and low-rank adapters.  Written pair by pair from the definitions in
include/bsg.h; test infrastructure only."""
from __future__ import annotations

import numpy as np

NONE, OUTSIDE = -1, -2


def rows_needed(T, k, G, align=1, cap=0):
    """Rows that hold every outcome of a sort."""
    return G * cap if cap else (T * k + min(G, T * k) * (align - 1) if G else 0)


def sort_tokens(ids, G, align=1, cap=0, rows=None):
    """(offsets, row_of, pair_of, row_group) of ids [T, k], one pair at a time."""
    ids = np.asarray(ids)
    T, k = ids.shape
    rows = rows_needed(T, k, G, align, cap) if rows is None else rows
    members = [[] for _ in range(G)]
    for p, g in enumerate(ids.reshape(-1)):
        if 0 <= g < G:
            members[g].append(p)
    row_of = np.full(T * k, NONE, np.int32)
    pair_of = np.full(rows, OUTSIDE, np.int32)
    row_group = np.full(rows, NONE, np.int32)
    counts, offsets, row = [], [0], 0
    for g in range(G):
        keep = members[g][:cap] if cap else members[g]
        start = g * cap if cap else row
        for i, p in enumerate(keep):
            row_of[p] = start + i
            pair_of[start + i] = p
            row_group[start + i] = g
        if not cap:
            row = start + -(-len(keep) // align) * align
            pair_of[start + len(keep):row] = NONE
        counts.append(len(keep))
        offsets.append(row)
    return (np.array(counts if cap else offsets, np.int32), row_of.reshape(T, k), pair_of,
            row_group)


def dispatch(X, row_of, pair_of, out):
    """out with token rows at row_of, zeros at padding rows; other rows as they were."""
    out = out.copy()
    out[pair_of == NONE] = 0
    for t, j in np.argwhere(row_of >= 0):
        out[row_of[t, j]] = X[t]
    return out


def combine(Y, row_of, W=None):
    """sum_j W[t, j] Y[row_of[t, j]] in fp64, and sum_j |W Y| (the scale of its error)."""
    T, k = row_of.shape
    out, mag = np.zeros((T, Y.shape[1])), np.zeros((T, Y.shape[1]))
    for t, j in np.argwhere(row_of >= 0):
        v = (1.0 if W is None else float(W[t, j])) * Y[row_of[t, j]].astype(np.float64)
        out[t] += v
        mag[t] += np.abs(v)
    return out, mag


def combine_backward(dO, Y, row_of, pair_of, W, dY):
    """(dY, dW, sum_h |dO Y|) in fp64; rows of dY that belong to no group as they were."""
    T, k = row_of.shape
    dY = dY.astype(np.float64)
    dY[pair_of == NONE] = 0
    dW, mag = np.zeros((T, k)), np.zeros((T, k))
    for t, j in np.argwhere(row_of >= 0):
        r = row_of[t, j]
        dY[r] = (1.0 if W is None else float(W[t, j])) * dO[t]
        if Y is not None:
            dW[t, j] = np.dot(dO[t], Y[r])
            mag[t, j] = np.dot(np.abs(dO[t]), np.abs(Y[r]))
    return dY, dW, mag


def lora(X, A, B, ids, scale=None, base=None):
    """base + scale[g] B[g] (A[g] x) per token in fp64, g = ids[t] (outside [0, G): none),
    and a bound on the library's error before the final rounding: fp32 sums of K terms on
    the matrix cores (two roundings a term), the intermediate held to 2^-16, fp32 sums of
    2r terms, one fp32 addition of base."""
    T, K = X.shape
    G, r, _ = A.shape
    N = B.shape[1]
    out = np.zeros((T, N)) if base is None else base.astype(np.float64).copy()
    err = np.zeros((T, N))
    u24 = 2.0 ** -24
    for t in range(T):
        g = int(ids[t])
        if not 0 <= g < G:
            continue
        s = 1.0 if scale is None else float(scale[g])
        u = A[g] @ X[t]
        eu = 2 * K * u24 * (np.abs(A[g]) @ np.abs(X[t]))
        d = s * (B[g] @ u)
        ab = np.abs(B[g])
        err[t] = abs(s) * (ab @ eu + (2.0 ** -16 + (4 * r + 4) * u24) * (ab @ (np.abs(u) + eu)))
        err[t] += 2 * u24 * (np.abs(out[t]) + np.abs(d))
        out[t] += d
    return out, err
