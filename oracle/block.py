"""fp64 definitions of the parts of a decoder block with layer norms, biased
linear layers, dropout and a gated feed-forward part (test infrastructure).

Written from the formulas, one element-wise expression each; gradients are
written out and pinned against finite differences in
tests/test_oracle_block.py. The dropout mask follows the published generator
(Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
2011) in Python integers' arithmetic on uint64 arrays, pinned by its authors'
known answers.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erfc = np.frompyfunc(math.erfc, 1, 1)


def _normal_cdf(z):
    return 0.5 * _erfc(np.asarray(z, dtype=np.float64) / -math.sqrt(2.0)).astype(np.float64)  # the lower tail keeps its digits


def act(z, kind):
    if kind == "none":
        return z * 1.0
    if kind == "relu":
        return np.where(z > 0, z, 0.0)
    if kind == "gelu":
        return z * _normal_cdf(z)
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1.0 + np.exp(-z))


def act_slope(z, kind):
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if kind == "gelu":
        return _normal_cdf(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + np.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def layernorm_fwd(x, g, b, eps):
    m = x.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(axis=1, keepdims=True) + eps)
    return (x - m) * r * g + b, m[:, 0], r[:, 0]


def layernorm_bwd(x, g, m, r, dy):
    xh = (x - m[:, None]) * r[:, None]
    w = dy * g
    dx = r[:, None] * (w - w.mean(axis=1, keepdims=True) - xh * (w * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def philox(counter, key):
    """Ten rounds of Philox4x32 on arrays of counters: counter four and key two
    uint32 values or arrays (held in uint64); returns the four words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def dropout_keep(rows, cols, p, seed, offset, row0=0):
    """True where element (t, j) is kept: word j % 4 of the block with counter
    (j / 4, row0 + t, offset) and key seed is at least p 2^32."""
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    q = np.arange((cols + 3) // 4)[None, :]
    t = row0 + np.arange(rows)[:, None]
    zero = np.zeros((rows, q.shape[1]), dtype=np.uint64)
    w = philox([q + zero, t.astype(np.uint64) + zero, zero + np.uint64(offset % 2 ** 32), zero + np.uint64(offset >> 32)],
               (seed % 2 ** 32, seed >> 32))
    words = np.stack(w, axis=2).reshape(rows, -1)[:, :cols]
    return words >= np.uint64(round(float(np.float32(p)) * 2 ** 32))


def drop(v, p, keep):
    """v / (1 - p) where kept, 0 elsewhere."""
    return np.where(keep, v / (1.0 - float(np.float32(p))), 0.0)


def linear_fwd(A, W, bias, kind, p=0.0, keep=None, R=0.0):
    """(C, U): U = A W^T + bias, C = R + drop(act(U))."""
    U = A @ W.T + bias
    C = act(U, kind)
    return R + (drop(C, p, keep) if p else C), U


def linear_bwd_act(dY, W, Z, kind, p=0.0, keep=None):
    """(dZ, db) from dY and the later layer's weight W [K, N]."""
    return act_bwd(dY @ W, Z, kind, p, keep)


def act_bwd(dC, Z, kind, p=0.0, keep=None):
    dZ = dC * act_slope(Z, kind)
    if p:
        dZ = drop(dZ, p, keep)
    return dZ, dZ.sum(axis=0)


def gated_fwd(x, Wg, Wu, kind):
    g, u = x @ Wg.T, x @ Wu.T
    return act(g, kind) * u, g, u


def gated_bwd(dy, Wd, g, u, kind):
    """(dgate, dup, h) from dy and the down projection Wd [K, F]."""
    dh = dy @ Wd
    return dh * u * act_slope(g, kind), dh * act(g, kind), act(g, kind) * u
