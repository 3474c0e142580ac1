"""Log-probabilities where logits over tau lie far from zero: a row's results
depend on the differences of its logits alone, whatever their size.  u = 2^-24;
with d the distance of a logit over tau from the row's largest, an exponent is off
by 3u of d (the difference, its product and the constant), and the rest as in
test_gpu_logprobs."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import logprobs as ref
from tests import test_gpu_logprobs as L

pytestmark = pytest.mark.gpu

U = L.U
INF = float("inf")


def far_rows(V, ld, z, base, seed):
    """Eight rows about `base`."""
    import torch as t
    r = t.Generator().manual_seed(seed)
    kind = L.types()[z]
    at = t.tensor(base, dtype=t.float64).to(kind).double()
    bits = t.finfo(kind).eps * abs(float(at)) / 2
    Z = t.full((8, ld), 0.0, dtype=t.float64)
    Z[0] = at
    Z[1] = at + t.randint(0, 4, (ld,), generator=r) * bits           # a few steps of the type apart
    Z[2] = at
    Z[2, ::3] = -INF                                                 # masked columns beside it
    Z[3] = at
    Z[3, V // 2] = at - 64 * bits
    Z[4] = t.randn(ld, generator=r).double() * 3                     # an ordinary row
    Z[5] = -INF
    Z[5, V - 1] = at                                                 # one column
    Z[6] = at
    Z[6, V - V // 5:V] = t.randn(V // 5, generator=r).double()       # ordinary ones come last
    Z[7] = at + t.randn(ld, generator=r).double() * abs(at) / 8      # all of them far apart
    most = t.finfo(kind).max
    target = t.randint(0, V, (8,), generator=r).to(t.int32)
    target[2], target[3], target[5] = V // 2 | 1 if (V // 2 | 1) % 3 and (V // 2 | 1) < V else 1, V // 2, V - 1
    Z = t.where(Z == -INF, Z, Z.clamp(-most, most))
    return Z.to(kind), target, t.randn(8, generator=r), t.randn(8, generator=r)


class Far:
    """The results in 64 bits, and what each may be off by before the output's rounding."""

    def __init__(self, Z, target, tau, V, g=None, h=None):
        z, at = Z.double().numpy(), target.numpy()
        g, h = (np.zeros(len(z)) if x is None else x.double().numpy() for x in (g, h))
        M = len(z)
        self.logp, self.entropy, self.lse, self.dZ = np.zeros(M), np.zeros(M), np.zeros(M), np.zeros_like(z)
        self.lim_logp, self.lim_entropy, self.lim_lse, self.lim_dZ = np.zeros(M), np.zeros(M), np.zeros(M), np.zeros_like(z)
        self.log_q, self.lim_log_q = np.zeros((M, V)), np.zeros((M, V))
        adds = V / 64 + 64
        for m in range(M):
            high = z[m, :V].max()
            d = (high - z[m, :V]) / np.float64(np.float32(tau))
            e = np.exp(-np.minimum(d, 1e4))
            s = e.sum()
            q, log_q, near = e / s, -d - np.log(s), np.where(e > 0, d, 0.0)
            mean = (q * near).sum()
            off_s = U * (4 + adds + 4 * mean)
            off = off_s + 8 * U * (np.log(V) + d)
            ent = mean + np.log(s)
            t = int(at[m])
            self.log_q[m], self.lim_log_q[m] = log_q, off
            self.logp[m], self.lim_logp[m] = log_q[t], off[t]
            self.lse[m] = high / np.float64(np.float32(tau)) + np.log(s)
            self.lim_lse[m] = off_s + 4 * U * (np.log(V) + 2 * abs(high) / tau + 1)
            self.entropy[m] = ent
            self.lim_entropy[m] = lim_e = off_s * (1 + mean) + U * (
                (8 + adds) * mean + 8 * (q * near ** 2).sum() + 8 * np.log(V) + 4)
            gm, hm = abs(g[m]), abs(h[m])
            own = np.zeros(V)
            own[t] = 1.0
            finite = np.where(q > 0, log_q, 0.0)
            dz = g[m] * (own - q) - h[m] * q * (finite + ent)
            size = gm + hm * (np.abs(finite) + abs(ent))
            off_q = np.where(q > 0, off, 0.0)
            lim = q * (off_q + 16 * U) * size + q * hm * (off_q + lim_e + 4 * U * (np.abs(finite) + abs(ent)))
            lim[t] += 4 * U * gm
            # an exponential below fp32's normal numbers is 0: 2^-126 of the row's largest, times its factor
            lim += 2.0 ** -126 * size
            self.dZ[m, :V] = dz / tau
            self.lim_dZ[m, :V] = lim / tau + 4 * U * np.abs(dz / tau)


def check(got, want, lim, kind, what):
    got = L.numpy(got)
    with np.errstate(invalid="ignore"):
        want = np.where(np.abs(want) > np.finfo(np.float32).max, np.sign(want) * INF, want)
        far = np.abs(got - want) - lim - L.HALF[kind] * (np.abs(want) + lim) - L.TINY[kind]
    far = np.where(got == want, -1.0, far)  # (equal infinities)
    assert not np.isnan(got).any(), f"{what}: NaN"
    at = np.unravel_index(np.argmax(far), far.shape)
    assert far[at] <= 0, f"{what}: {got[at]} for {want[at]} at {at}, {far[at]:.3e} past its bound"


# forms of the kernel: chunks in registers of 512 or 1,024 threads, and rows read again
FORMS = [("bf16", 700, 700), ("f32", 1003, 1008), ("bf16", 9000, 9003), ("f32", 20011, 20011), ("f16", 40001, 40008),
         ("f32", 50001, 50008), ("bf16", 140000, 140000)]
BASES = {"bf16": (-1e9, -1e10, -9e29, 1e10, 3e7, 3e38, 700.0, -1e4, 2.26e4, 2.28e4),
         "f32": (-1e9, -1e10, -9e29, 1e10, -1.7e7, 3e9, 5000.0), "f16": (-65504.0, 65504.0, -60000.0, 150.0)}


@pytest.mark.parametrize("z,V,ld", FORMS)
@pytest.mark.parametrize("tau", [1.0, 0.1, 1e-5])
def test_forward(z, V, ld, tau):
    import torch as t
    for base in BASES[z]:
        print(f"far logprobs {z} {V} base={base} tau={tau}", flush=True)
        Z, target, g, h = far_rows(V, ld, z, base, seed=V)
        g, h = g * tau, h * tau  # (gradients that every type holds)
        b = Far(Z, target, tau, V, g, h)
        out = L.forward(Z, target, tau, V, 5, g, h)
        check(out["logp"], b.logp, b.lim_logp, "f32", "logp")
        check(out["entropy"], b.entropy, b.lim_entropy, "f32", "entropy")
        held = np.abs(b.lse) < 3.4e38
        check(out["lse"][t.from_numpy(held).cuda()], b.lse[held], b.lim_lse[held], "f32", "lse")
        check(out["dZ"], b.dZ, b.lim_dZ, z, "dZ")
        top = ref.top(L.numpy(Z), 5, V)
        np.testing.assert_array_equal(out["top_index"].cpu().numpy(), top)
        for m in range(8):
            n = (top[m] >= 0).sum()
            check(out["top_logp"][m, :n], b.log_q[m, top[m, :n]], b.lim_log_q[m, top[m, :n]], "f32", "top")
        bg = Far(Z, target, tau, V, g)
        likelihood = L.forward(Z, target, tau, V, 0, g, None, in_place=True)
        check(likelihood["dZ"], bg.dZ, bg.lim_dZ, z, "dZ of the likelihood")


@pytest.mark.parametrize("z,V,ld", FORMS)
@pytest.mark.parametrize("tau", [1.0, 0.1, 1e-5])
def test_backward(z, V, ld, tau):
    """From the saved sums.  fp32 holds a log-sum-exp of 65536 and more in steps of 2^-7 and
    more; those rows find their sum again, the others count from the lse they are given."""
    import torch as t
    for base in BASES[z]:
        print(f"far logprobs backward {z} {V} base={base} tau={tau}", flush=True)
        Z, target, g, h = far_rows(V, ld, z, base, seed=V + 1)
        g, h = g * tau, h * tau
        target[4] = -100
        h[3] = 0.0
        target[6] = -1 if V % 2 else target[6]
        out = L.forward(Z, target, tau, V)
        lse, entropy = out["lse"].cpu(), out["entropy"].cpu()
        far = lse.abs().numpy() >= 65536
        gone = ((target < 0) & (h == 0)).numpy()
        for dl, de in ((g, None), (None, h), (g, h)):
            with_target = t.where(target < 0, 0, target)
            own = None if dl is None else t.where(target < 0, 0.0, dl)
            b = Far(Z, with_target, tau, V, own, de)
            if (~far).any():
                n = L.Bounds(Z[~far], target[~far], float(np.float32(tau)), V, None if dl is None else dl[~far],
                             None if de is None else de[~far], lse[~far], entropy[~far])
                b.dZ[~far] = n.dZ
                # (an exponential below fp32's normal numbers is 0: 2^-126 times its factor, log q of -88 in it)
                size = sum(np.abs(x.numpy()) * y for x, y in ((dl, 1), (de, 100)) if x is not None) / tau
                b.lim_dZ[~far] = n.lim_dZ + 2.0 ** -126 * size[~far, None]
            got = L.backward(Z, target, tau, V, lse, entropy, dl, de)
            check(got, b.dZ, b.lim_dZ, z, "dZ")
            assert not L.numpy(got)[gone].any()
            assert t.equal(L.backward(Z, target, tau, V, lse, entropy, dl, de, in_place=True), got)


def test_a_saved_lse_past_fp32():
    """A logit over tau that fp32 does not hold: its lse is infinite, the gradient the differences'."""
    import torch as t
    Z, target, g, h = far_rows(5000, 5000, "f32", 3e36, seed=1)
    tau = 1e-4
    g, h = g * tau, h * tau
    b = Far(Z, target, tau, 5000, g, h)
    out = L.forward(Z, target, tau, 5000, 0, g, h)
    check(out["dZ"], b.dZ, b.lim_dZ, "f32", "dZ")
    lse = out["lse"].cpu()
    assert (lse == INF).any()
    got = L.backward(Z, target, tau, 5000, lse, out["entropy"].cpu(), g, h)
    rows = (lse.abs() >= 65536).numpy()
    check(got[t.from_numpy(rows).cuda()], b.dZ[rows], b.lim_dZ[rows], "f32", "dZ from the saved sums")


@pytest.mark.parametrize("z,V,ld", [FORMS[0], FORMS[5]])
def test_not_a_number_in_far_rows(z, V, ld):
    import torch as t
    Z, target, g, h = far_rows(V, ld, z, -1e10, seed=3)
    Z[0, 5], Z[1, V // 2], Z[7, V - 1] = float("nan"), INF, float("nan")
    out = L.forward(Z, target, 1.0, V, 4, g, h)
    lse, entropy = out["lse"].cpu(), out["entropy"].cpu()
    want = [m in (0, 1, 7) for m in range(8)]
    back = L.backward(Z, target, 1.0, V, lse, entropy, g, h)
    for x in (out["lse"], out["entropy"], out["logp"]):
        assert x.isnan().tolist() == want
    given = lse.clone()
    given[[0, 1, 7]] = -1e10                # a number, of another pass over the logits
    other = L.backward(Z, target, 1.0, V, given, t.nan_to_num(entropy), g, h)
    for x in (out["dZ"], back, other):
        assert x[:, :V].isnan().all(1).tolist() == want and x.isnan().any(1).tolist() == want
        assert not x[:, V:].any()
