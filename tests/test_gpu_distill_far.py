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
            if (log_q[p > 2.0 ** -149] < -np.finfo(np.float32).max).any():
                self.loss[m] = INF
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
        print(f"far distill {z} {V} base={base} tau={tau}", flush=True)
        Z, T, at, w = draw(V, ld, z, base, 30, seed=V)
        w = w / tau                 # (gradients that every type holds)
        b = Far(Z, T, at, tau, w, V)
        loss, lse, dZ = D.call(Z, T, at, tau, w, V)
        F.check(lse, b.lse, b.lim_lse, "f32", "lse")
        F.check(dZ, b.dZ, b.lim_dZ, z, "dZ")
        F.check(loss, b.loss, b.lim_loss, "f32", "loss")


@pytest.mark.parametrize("z,V,ld", F.FORMS)
@pytest.mark.parametrize("tau", [1.0, 0.1, 1e-5])
def test_gradient_from_the_saved_sum(z, V, ld, tau):
    """fp32 holds a log-sum-exp of 65536 and more in steps of 2^-7 and more; those rows find
    their sum again, the others count from the lse they are given."""
    import torch as t
    for base in F.BASES[z]:
        print(f"far distill from lse {z} {V} base={base} tau={tau}", flush=True)
        Z, T, at, w = draw(V, ld, z, base, 30, seed=V + 1)
        at[3] = -1                  # no entries
        w = w / tau
        lse = D.call(Z, T, at, tau, w, V)[1]
        b = Far(Z, T, at, tau, w, V)
        near = (lse.abs().cpu() < 65536).numpy()
        if near.any():
            with np.errstate(over="ignore"):
                (_, _, dz), lim = D.bounds(Z[near], T[near], at[near], float(np.float32(tau)), w[near], V,
                                           lse.cpu()[near].numpy())
            # (an exponential below fp32's normal numbers is 0)
            b.dZ[near], b.lim_dZ[near] = dz, lim[2] + 2.0 ** -126 * w[near, None].numpy() * tau
        d = [x.cuda() for x in (Z, T, at, w)]
        dZ = t.full_like(d[0], float("nan"))
        q.qlora_distill_bwd(d[0], d[1], d[2], tau, lse, d[3], dZ, vocab=V)
        F.check(dZ, b.dZ, b.lim_dZ, z, "dZ from lse")
        assert not dZ[1].any() and not dZ[3].any()
        q.qlora_distill_bwd(d[0], d[1], d[2], tau, lse, d[3], d[0], vocab=V)
        assert t.equal(d[0], dZ)


@pytest.mark.parametrize("z,V,ld", [F.FORMS[0], F.FORMS[5]])
def test_not_a_number_in_far_rows(z, V, ld):
    import torch as t
    Z, T, at, w = draw(V, ld, z, -1e10, 12, seed=3)
    Z[0, 5], Z[3, V // 2], Z[6, V - 1] = float("nan"), INF, float("nan")
    want = [m in (0, 3, 6) for m in range(8)]
    loss, lse, dZ = D.call(Z, T, at, 1.0, w, V)
    assert loss.isnan().tolist() == want and lse.isnan().tolist() == want
    given = lse.clone()
    given[[0, 3, 6]] = -1e10       # a number, of another pass over the logits
    d = [x.cuda() for x in (Z, T, at, w)]
    for saved in (lse, given):
        back = t.full_like(d[0], 7.0)
        q.qlora_distill_bwd(d[0], d[1], d[2], 1.0, saved, d[3], back, vocab=V)
        for x in (dZ, back):
            assert x[:, :V].isnan().all(1).tolist() == want and x.isnan().any(1).tolist() == want
            assert not x[:, V:].any()
