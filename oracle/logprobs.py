"""fp64 reference of the log-probabilities of given tokens, row by row from the
definition.  Oracle (test infrastructure only; see ``oracle/__init__``).

Per token, z its logits, q = softmax(z/tau) over V columns, t the given column
(outside [0, V): no token):

  logp = log q_t, entropy = −Σ_v q_v·log q_v, lse = log Σ_v exp(z_v/tau)
  dZ[v] = (g·([v = t] − q_v) − h·q_v·(log q_v + entropy))/tau

A logit of −infinity has q = 0.  A row whose largest logit is below -1e30 has no
columns: logp, entropy and gradient 0, lse −infinity.  A token of g = h = 0 has a
zero gradient whatever its logits.  NaN where the formulas have it.
"""

from __future__ import annotations

import math

import numpy as np


def logprobs(Z, target, tau, vocab=None, g=None, h=None, lse=None, entropy=None):
    """(logp [M], lse [M], entropy [M], dZ [M, ldz]); lse, entropy: take them as given for dZ."""
    Z = np.asarray(Z, dtype=np.float64)
    M, ldz = Z.shape
    V = ldz if vocab is None else vocab
    logp, out_lse, out_ent, dZ = np.zeros(M), np.zeros(M), np.zeros(M), np.zeros((M, ldz))
    for m in range(M):
        t = int(target[m])
        has = 0 <= t < V
        z = Z[m, :V] / tau
        high = np.fmax.reduce(z)
        bad = np.isnan(z).any() or high == math.inf
        if bad:
            out_lse[m] = out_ent[m] = math.nan
            logp[m] = math.nan if has else 0.0
            log_q = np.full(V, math.nan)
        elif high * tau < -1e30:
            out_lse[m] = -math.inf
            continue
        else:
            log_s = math.log(math.fsum(np.exp(z - high)))
            log_q = (z - high) - log_s
            q = np.exp(log_q)
            out_lse[m] = high + log_s
            out_ent[m] = math.fsum(-q[q > 0] * log_q[q > 0])
            logp[m] = log_q[t] if has else 0.0
        use, ent = out_lse[m], out_ent[m]
        if lse is not None:
            use = float(lse[m])
            if use == -math.inf:
                continue
            log_q = z - use
        if entropy is not None:
            ent = float(entropy[m])
        gm = float(g[m]) if g is not None and has else 0.0
        hm = float(h[m]) if h is not None else 0.0
        if gm == 0.0 and hm == 0.0:
            continue
        with np.errstate(invalid="ignore"):
            q = np.exp(log_q)
            d = -gm * q
            if hm != 0.0:
                d = d - hm * q * (np.where(q == 0, 0.0, log_q) + ent)
        if gm != 0.0:
            d[t] += gm
        dZ[m, :V] = d / tau
    return logp, out_lse, out_ent, dZ


def top(Z, k, vocab=None):
    """The k columns of the largest logits of every row, equal ones by their index (int [M, k]; -1 where a row has
    fewer; NaN and logits below -1e30 are never among them)."""
    Z = np.asarray(Z, dtype=np.float64)
    V = Z.shape[1] if vocab is None else vocab
    out = np.full((Z.shape[0], k), -1, np.int64)
    for m, row in enumerate(Z[:, :V]):
        at = np.flatnonzero(row > -1e30)
        at = at[np.argsort(-row[at], kind="stable")][:k]
        out[m, :len(at)] = at
    return out
