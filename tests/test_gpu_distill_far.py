"""Distillation where the student's logits over tau lie far from zero: loss and
gradient depend on the differences of a row's logits alone, whatever their size.
u = 2^-24; with d the distance of a logit over tau from the row's largest, an
exponent is off by 3u of d and the rest as in test_gpu_distill."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from tests import test_gpu_distill as D
from tests import test_gpu_logprobs_far as F

pytestmark = pytest.mark.gpu

U = D.U
INF = float("inf")


def draw(V, ld, z, base, k, seed):
    import torch as t
    r = t.Generator().manual_seed(seed)
    Z, _, _, _ = F.far_rows(V, ld, z, base, seed)
    at = t.stack([t.randperm(V, generator=r)[:k] for _ in range(8)]).to(t.int32)
    T, w = t.randn(8, k, generator=r) * 3, t.rand(8, generator=r) + 0.25
    # (an entry at a masked column has an infinite loss: row 2's and row 5's are columns)
    at[2] = at[2] // 3 * 3 + 1
    at[2] = t.where(at[2] < V, at[2], 1)
    at[5] = V - 1
    w[1] = 0.0
    at[7, 1:] = -1
    return Z, T, at, w


class Far:
    def __init__(self, Z, T, at, tau, w, V):
        z, tt, a, w = Z.double().numpy(), T.double().numpy(), at.numpy(), w.double().numpy()
        M, k = tt.shape
        tau32 = np.float64(np.float32(tau))
        self.loss, self.lse, self.dZ = np.zeros(M), np.zeros(M), np.zeros_like(z)
        self.lim_loss, self.lim_lse, self.lim_dZ = np.zeros(M), np.zeros(M), np.zeros_like(z)
        adds = V / 64 + 64
        for m in range(M):
            high = z[m, :V].max()
            d = (high - z[m, :V]) / tau32
            e = np.exp(-np.minimum(d, 1e4))
            s = e.sum()
            qv, near = e / s, np.where(e > 0, d, 0.0)
            off_s = U * (4 + adds + 4 * (qv * near).sum())
            self.lse[m] = high / tau32 + np.log(s)
            self.lim_lse[m] = off_s + 4 * U * (np.log(V) + 2 * abs(high) / tau + 1)
            ok = (a[m] >= 0) & (a[m] < V)
            if not ok.any() or w[m] == 0:
                continue
            y = tt[m][ok] / tau32
            y = y - y.max()
            log_p = y - np.log(np.exp(y).sum())
            p = np.exp(log_p)
            off_p = p * U * (16 + 8 * -y + k)
            log_q = -d[a[m][ok]] - np.log(s)
            off_q = off_s + 8 * U * (np.log(V) + d[a[m][ok]])
            gap = np.abs(log_p - log_q)
            self.loss[m] = w[m] * tau32 ** 2 * (p * (log_p - log_q)).sum()
            self.lim_loss[m] = w[m] * tau ** 2 * (
                (p * (off_q + U * (8 * np.abs(log_p) + 8 * np.abs(log_q) + 8 * -y.min() + k))).sum()
                + (off_p * gap).sum() + U * (k + 8) * (p * gap).sum())
            dz = qv.copy()
            np.add.at(dz, a[m][ok], -p)
            # (an exponential below fp32's normal numbers is 0: 2^-126 of the row's largest)
            lim = qv * (off_s + U * (16 + 8 * near)) + 2.0 ** -126
            np.add.at(lim, a[m][ok], off_p + p * U * 4)
            self.dZ[m, :V] = w[m] * tau * dz
            self.lim_dZ[m, :V] = w[m] * tau * lim + 4 * U * np.abs(w[m] * tau * dz)


@pytest.mark.parametrize("z,V,ld", F.FORMS)
@pytest.mark.parametrize("tau", [1.0, 0.1, 1e-5])
def test_loss_and_gradient(z, V, ld, tau):
    for base in F.BASES[z]:
        if abs(base) / tau > 3e38:  # (out of the documented range)
            continue
        print(f"far distill {z} {V} base={base} tau={tau}", flush=True)
        Z, T, at, w = draw(V, ld, z, base, 30, seed=V)
        w = w / tau                 # (gradients that every type holds)
        b = Far(Z, T, at, tau, w, V)
        loss, lse, dZ = D.call(Z, T, at, tau, w, V)
        F.check(lse, b.lse, b.lim_lse, "f32", "lse")
        F.check(dZ, b.dZ, b.lim_dZ, z, "dZ")
        F.check(loss, b.loss, b.lim_loss, "f32", "loss")
