"""fp64 reference of the distillation loss against a teacher's top logits, row
by row from the definition.  Oracle (test infrastructure only; see
``oracle/__init__``).

Per token, z the student's logits, (t_i, c_i) the teacher's top logits and
their columns (outside [0, V): no entry):

  p = softmax(t/tau) over the entries, q = softmax(z/tau) over the columns
  loss = w·tau²·Σ_i p_i·(log p_i − log q_{c_i})
  dZ[v] = w·tau·(q_v − Σ_{i: c_i = v} p_i)

Zero for a token of weight 0, without entries, or whose largest logit is below
-1e30 (every column masked; its lse is −infinity).  NaN where the formulas have
it: a NaN or +infinity among the logits, or among the entries' logits.
"""

from __future__ import annotations

import math

import numpy as np


def distill(Z, top, at, tau, weight=None, vocab=None, lse=None):
    """(loss [M], lse [M], dZ [M, ldz]); lse: take it as given for dZ."""
    Z, top = np.asarray(Z, dtype=np.float64), np.asarray(top, dtype=np.float64)
    M, ldz = Z.shape
    V = ldz if vocab is None else vocab
    loss, out_lse, dZ = np.zeros(M), np.zeros(M), np.zeros((M, ldz))
    for m in range(M):
        w = 1.0 if weight is None else float(weight[m])
        z = Z[m, :V] / tau
        high = z.max()
        if high * tau <= -1e30:
            out_lse[m] = -math.inf
            continue
        out_lse[m] = high + math.log(math.fsum(np.exp(z - high)))
        use = out_lse[m] if lse is None else float(lse[m])
        entries = [(top[m, i] / tau, int(at[m, i])) for i in range(top.shape[1])
                   if 0 <= at[m, i] < V and top[m, i] != -math.inf]
        if not entries or w == 0.0 or use == -math.inf:
            continue
        t_high = max(t for t, _ in entries)
        t_log = math.log(math.fsum(math.exp(t - t_high) for t, _ in entries))
        dZ[m, :V] = np.exp(z - use)
        for t, c in entries:
            log_p = (t - t_high) - t_log  # (not t - (t_high + t_log): the logits may be huge)
            p = math.exp(log_p)
            if p != 0.0:
                loss[m] += p * (log_p - (z[c] - use))
            dZ[m, c] -= p
        loss[m] *= w * tau * tau
        dZ[m] *= w * tau
    return loss, out_lse, dZ
