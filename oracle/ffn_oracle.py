"""Plain CPU definitions, in 64 bits, of the 4-bit group-scaled linear and the gated feed-forward
block with its 8-bit checkpoint and its backward pass.  numpy only; shares no code with the GPU
path.

  int4:     w[n,k] = (q[n,k] - z[n,k//group]) * s[n,k//group], element 2i in the low nibble of byte i
  forward:  g = x Wg^T, u = x Wu^T, h = silu(a min(g, L)) * clamp(u, -L, L)
  backward: du = dh silu(a g') [|u| <= L], dg = dh u' a silu'(a g') [g <= L], g' = min(g, L),
            u' = clamp(u, -L, L); dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
"""
from __future__ import annotations

import numpy as np

CKPT_GROUP = 128


def int4_unpack(w, K):
    """uint8 [N, >=K/2] -> codes 0..15 as float64 [N, K]."""
    q = np.empty((w.shape[0], K), np.float64)
    q[:, 0::2] = w[:, :K // 2] & 15
    q[:, 1::2] = w[:, :K // 2] >> 4
    return q


def int4_dequant(w, s, z, K, group):
    """s: float64 [N, ceil(K/group)]; z: uint8 likewise, or None for 8."""
    at = np.arange(K) // group
    zero = 8.0 if z is None else z.astype(np.float64)[:, at]
    return (int4_unpack(w, K) - zero) * s[:, at]


def linear(x, w):
    """(y, sum |x w|) in float64."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def sigmoid(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


def silu(t):
    return t * sigmoid(t)


def gated(g, u, alpha=1.0, limit=np.inf):
    return silu(alpha * np.minimum(g, limit)) * np.clip(u, -limit, limit)


def gated_grad(dh, g, u, alpha=1.0, limit=np.inf):
    """(dg, du)."""
    t = alpha * np.minimum(g, limit)
    s = sigmoid(t)
    dg = dh * np.clip(u, -limit, limit) * alpha * (s + t * s * (1.0 - s))
    return np.where(g <= limit, dg, 0.0), np.where(np.abs(u) <= limit, dh * t * s, 0.0)


def checkpoint_int8(v):
    """(codes, scale [M, ceil(I/128)]): scale = max|v| / 127, codes = round_half_even(v / scale)."""
    M, I = v.shape
    groups = -(-I // CKPT_GROUP)
    codes, scale = np.zeros((M, I)), np.zeros((M, groups))
    for j in range(groups):
        part = v[:, j * CKPT_GROUP:(j + 1) * CKPT_GROUP]
        s = np.abs(part).max(axis=1) / 127.0
        scale[:, j] = s
        codes[:, j * CKPT_GROUP:(j + 1) * CKPT_GROUP] = np.rint(part / np.where(s > 0, s, 1.0)[:, None])
    return codes, scale


def checkpoint_values(codes, scale):
    return codes * np.repeat(scale, CKPT_GROUP, axis=1)[:, :codes.shape[1]]


def backward(dh, x, w13, g, u, alpha=1.0, limit=np.inf):
    """(dx, dw13, dgu) from the checkpoint's values g and u."""
    dg, du = gated_grad(dh, g, u, alpha, limit)
    dgu = np.concatenate([dg, du], axis=1)
    return dgu @ w13, dgu.T @ x, dgu
