"""fp64 references of the linear layer with dropout of its adapter's input and of
the gated feed-forward block, from the formulas.  Oracle (test infrastructure
only; see ``oracle/__init__``).

  Y = X·Ŵᵀ + s·T·Bᵀ,  T = D(X)·Aᵀ,  D(X) = keep*X
  V = dY·B,  dX = dY·Ŵ + s·keep*(V·A),  dA = s·Vᵀ·D(X),  dB = s·dYᵀ·T
  gated: H = act(G)*U, G and U two such layers of one X and one keep;
  dG = RNE_bf16(fl32(dH·U·act'(G))), dU = RNE_bf16(fl32(dH·act(G)))

keep_i = 65536/(65536 − t) where the 16 bits of element i are at least t =
round(65536·p), else 0; the bits are those of the counter-based generator
Philox4x32-10 (Salmon, Moraes, Dror and Shaw 2011) for the key `seed` and the
counter (i // 8, offset).

Every product takes an ``absolute`` flag: with the absolute values of all inputs
it returns the sums of absolute terms that rounding bounds need.
"""

from __future__ import annotations

import math

import numpy as np

LOW = (1 << 32) - 1


def philox4x32(counter, key, rounds=10):
    """One block: four 32-bit words from four and a key of two (plain integers)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & LOW, (a >> 32) ^ c[3] ^ k[1], a & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


def pieces(M, K, seed, offset):
    """The 16 bits of every element of X [M, K] (uint16)."""
    n = -(-M * K // 8)
    i = np.arange(n, dtype=np.uint64)
    low = np.uint64(LOW)
    c = [i & low, i >> np.uint64(32), np.full(n, offset & LOW, np.uint64), np.full(n, (offset >> 32) & LOW, np.uint64)]
    k = [seed & LOW, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    words = np.stack(c, 1).astype(np.uint32)
    return np.stack((words & 0xFFFF, words >> 16), 2).astype(np.uint16).reshape(-1)[:M * K].reshape(M, K)


def keep(M, K, p, seed, offset=0):
    """What each element of X is multiplied with."""
    t = round(65536 * p)
    if t == 0:
        return np.ones((M, K))
    return (pieces(M, K, seed, offset) >= t) * (65536 / (65536 - t))


def _inputs(absolute, *arrays):
    out = [np.asarray(a, dtype=np.float64) for a in arrays]
    return [np.abs(a) for a in out] if absolute else out


def _dropped(X, mask):
    return np.where(mask != 0, X, 0.0) * mask  # (a dropped NaN is gone)


def forward(X, W_hat, A, B, s, mask, absolute=False):
    """(Y, T)"""
    X, W_hat, A, B = _inputs(absolute, X, W_hat, A, B)
    T = _dropped(X, mask) @ A.T
    return X @ W_hat.T + abs(s) * (T @ B.T) if absolute else X @ W_hat.T + s * (T @ B.T), T


def backward(X, dY, W_hat, A, B, s, mask, T=None, absolute=False):
    """(dX, dA, dB); T: the saved low-rank factor, recomputed when None."""
    X, dY, W_hat, A, B = _inputs(absolute, X, dY, W_hat, A, B)
    s = abs(s) if absolute else s
    if T is None:
        T = _dropped(X, mask) @ A.T
    else:
        (T,) = _inputs(absolute, T)
    V = dY @ B
    return dY @ W_hat + s * _dropped(V @ A, mask), s * (V.T @ _dropped(X, mask)), s * (dY.T @ T)


def act(kind, g):
    """act(g) and act'(g)."""
    g = np.asarray(g, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "silu":
            h, slope = g, 1.0
        else:
            c = 2 * math.sqrt(2 / math.pi)
            h, slope = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
        s, rest = 1 / (1 + np.exp(-h)), 1 / (1 + np.exp(h))
        return g * s, s * (1 + np.where(rest == 0, 0.0, g * rest * slope))


def bf16(v):
    """fp64 → fp32 → bf16, each to nearest even, as fp64."""
    with np.errstate(over="ignore"):
        f = np.asarray(v, dtype=np.float64).astype(np.float32)
    u = f.view(np.uint32)
    r = ((u + (0x7FFF + ((u >> np.uint32(16)) & np.uint32(1))).astype(np.uint32)) & np.uint32(0xFFFF0000)).view(np.float32)
    return np.where(np.isfinite(f), r, f).astype(np.float64)


def gate_gradients(kind, G, U, dH):
    """(dG, dU), rounded to bf16."""
    value, slope = act(kind, G)
    U, dH = np.asarray(U, dtype=np.float64), np.asarray(dH, dtype=np.float64)
    return bf16(dH * U * slope), bf16(dH * value)
