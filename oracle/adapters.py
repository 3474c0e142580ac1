"""fp64 references of the linear layer whose tokens carry different low-rank
adapters, token by token from the formulas.  Oracle (test infrastructure only;
see ``oracle/__init__``).

P1 §七 (dataflow figure): one frozen base, the adapter's path added to its
output; with several adapters a(m) picks the one of token m (outside
[0, count): none):

  Y[m] = X[m]·Ŵᵀ + s_a·(X[m]·A_aᵀ)·B_aᵀ,   T[m] = X[m]·A_aᵀ
  U[m] = dY[m]·B_a,   dX[m] = dY[m]·Ŵ + s_a·U[m]·A_a
  dA_a = s_a·Σ_m U[m]ᵀ·X[m],   dB_a = s_a·Σ_m dY[m]ᵀ·T[m]

Every function takes an ``absolute`` flag: with the absolute values of all
inputs it returns the sums of absolute terms that rounding bounds need.
"""

from __future__ import annotations

import numpy as np


def _inputs(absolute, *arrays):
    out = [np.asarray(a, dtype=np.float64) for a in arrays]
    return [np.abs(a) for a in out] if absolute else out


def _adapter(index, m, count):
    a = int(index[m])
    return a if 0 <= a < count else None


def forward(X, W_hat, A, B, scale, index, absolute=False):
    """(Y, T): A [count, r, K], B [count, N, r], scale [count], index [M]."""
    X, W_hat, A, B, scale = _inputs(absolute, X, W_hat, A, B, scale)
    Y = X @ W_hat.T
    T = np.zeros((X.shape[0], A.shape[1]))
    for m in range(X.shape[0]):
        a = _adapter(index, m, len(scale))
        if a is not None:
            T[m] = A[a] @ X[m]
            Y[m] += scale[a] * (B[a] @ T[m])
    return Y, T


def backward(X, dY, W_hat, A, B, scale, index, T=None, absolute=False):
    """(dX, dA, dB); T: the saved low-rank factor, recomputed when None."""
    X, dY, W_hat, A, B, scale = _inputs(absolute, X, dY, W_hat, A, B, scale)
    if T is None:
        T = forward(X, W_hat, A, B, scale, index)[1]
    else:
        (T,) = _inputs(absolute, T)
    dX = dY @ W_hat
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for m in range(X.shape[0]):
        a = _adapter(index, m, len(scale))
        if a is not None:
            U = dY[m] @ B[a]
            dX[m] += scale[a] * (U @ A[a])
            dA[a] += scale[a] * np.outer(U, X[m])
            dB[a] += scale[a] * np.outer(dY[m], T[m])
    return dX, dA, dB
