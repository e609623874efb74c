"""Plain CPU definitions, in 64 bits, of the mixture-of-experts layers on bf16, 8-bit and 4-bit weights
and of the linear on 8-bit codes.  numpy only; shares no code with the GPU path.

  pair (m, j) with expert e = ids[m, j] (left out if e is outside [0, E)):
    g = W13[e][:I] x_m, u = W13[e][I:] x_m, h = silu(a min(g, L)) * clamp(u, -L, L)
    y_m = sum_j weights[m, j] W2[e] h_(m, j)
  codes: scale = max|v| / 127, code = v / scale rounded half to even, in fp32 (a quotient of two fp32 values
  that is rounded to 64 bits first rounds to fp32 as if at once: 53 >= 2 * 24 + 2)
"""
from __future__ import annotations

import numpy as np

from .ffn_oracle import sigmoid


def codes(v):
    """(codes, scale) of the rows of bf16 values: scale and quotient are fp32, rounded once each."""
    scale = (np.abs(v).max(axis=-1, keepdims=True) / 127.0).astype(np.float32)
    q = (v / np.where(scale > 0, scale, 1.0).astype(np.float64)).astype(np.float32)
    return np.where(scale > 0, np.clip(np.rint(q.astype(np.float64)), -127, 127), 0.0), scale.astype(np.float64)


def gate_up(x, w13, ids):
    """(g, u, sum|x w| of both) of every pair [M * topk, I]; zeros where the id is outside [0, E)."""
    E, rows, _ = w13.shape
    out = np.zeros((2, ids.size, rows))
    for p, e in enumerate(ids.reshape(-1)):
        if 0 <= e < E:
            m = p // ids.shape[1]
            out[0, p] = w13[e] @ x[m]
            out[1, p] = np.abs(w13[e]) @ np.abs(x[m])
    I = rows // 2
    return out[0, :, :I], out[0, :, I:], out[1, :, :I], out[1, :, I:]


def activation(g, u, dg, du, alpha=1.0, limit=np.inf):
    """(h, how far it may be off) for g and u that are off by at most dg and du.  |d silu(a g)/dg| <=
    1.1 a; the exponential (2 + |1.16 t| ulp at |t| < 64) and the quotient put 2^-17 on h."""
    gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit)
    s = alpha * gc * sigmoid(alpha * gc)
    h = s * uc
    return h, 1.1 * abs(alpha) * dg * (np.abs(uc) + du) + np.abs(s) * du + 2.0 ** -17 * np.abs(h)


def down(h, w2, ids, weights):
    """(y, sum of magnitudes) [M, H] from h [M * topk, I]."""
    M, topk = ids.shape
    y, a = np.zeros((M, w2.shape[1])), np.zeros((M, w2.shape[1]))
    for p, e in enumerate(ids.reshape(-1)):
        if 0 <= e < w2.shape[0]:
            m, j = divmod(p, topk)
            y[m] += weights[m, j] * (w2[e] @ h[p])
            a[m] += abs(weights[m, j]) * (np.abs(w2[e]) @ np.abs(h[p]))
    return y, a


def linear_codes(xq, xs, w, ws):
    """(acc int64, acc xs ws in float64)."""
    acc = xq.astype(np.int64) @ w.astype(np.int64).T
    return acc, acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
