"""Log-probabilities, entropies, the most likely tokens and their gradient
against the fp64 oracle.  Bounds per element, u = 2^-24: an exponent is off by 2u
of itself (its constant and its one rounding), an exponential by that and 2u, a
row's sums by the additions of one thread and of the reduction, the output by
half a step of its type."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import logprobs as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}


def types():
    import torch as t
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}


def rows(M, V, ld, z, seed=0, scale=3.0):
    import torch as t
    r = t.Generator().manual_seed(seed)
    Z = (t.randn(M, ld, generator=r) * scale).to(types()[z])
    target = t.randint(0, V, (M,), generator=r).to(t.int32)
    return Z, target, t.randn(M, generator=r), t.randn(M, generator=r)


def nan(*shape, dtype=None):
    import torch as t
    return t.full(shape, float("nan"), device="cuda", dtype=dtype or t.float32)


def forward(Z, target, tau, V, k=0, g=None, h=None, in_place=False, stats=True):
    """{"logp", "lse", "entropy", "top_logp", "top_index", "dZ"}"""
    import torch as t
    M = Z.shape[0]
    d = [None if x is None else x.cuda() for x in (Z, target, g, h)]
    out = {"logp": nan(M), "lse": nan(M) if stats else None, "entropy": nan(M) if stats else None,
           "top_logp": nan(M, k) if k else None,
           "top_index": t.full((M, k), -7, dtype=t.int32, device="cuda") if k else None,
           "dZ": None if g is None and h is None else d[0] if in_place else nan(*Z.shape, dtype=Z.dtype)}
    q.qlora_logprobs_fwd(d[0], d[1], tau, d_logp=d[2], d_entropy=d[3], vocab=V, **out)
    return out


def backward(Z, target, tau, V, lse, entropy, g, h, in_place=False):
    d = [None if x is None else x.cuda() for x in (Z, target, lse, entropy, g, h)]
    dZ = d[0] if in_place else nan(*Z.shape, dtype=Z.dtype)
    q.qlora_logprobs_bwd(d[0], d[1], tau, d[2], d[4], dZ, entropy=d[3], d_entropy=d[5], vocab=V)
    return dZ


def numpy(x):
    return None if x is None else x.double().cpu().numpy()


class Bounds:
    """The oracle's values, and what each may be off by before the output's rounding."""

    def __init__(self, Z, target, tau, V, g=None, h=None, lse=None, entropy=None):
        z, at = numpy(Z), target.numpy()
        g, h, lse, entropy = numpy(g), numpy(h), numpy(lse), numpy(entropy)
        self.logp, self.lse, self.entropy, self.dZ = ref.logprobs(z, at, tau, V, g, h, lse, entropy)
        M = len(z)
        self.lim_logp, self.lim_lse, self.lim_entropy = np.zeros(M), np.zeros(M), np.zeros(M)
        self.lim_dZ, self.log_q = np.zeros_like(z), np.full((M, V), -np.inf)
        adds = V / 64 + 64  # additions of one thread (at least 64 of them share a row) and of the reduction
        for m in range(M):
            if self.lse[m] == -np.inf:
                continue
            x = z[m, :V] / tau
            x = np.maximum(x, x.max() - 1e4)
            use = self.lse[m] if lse is None else lse[m]
            ent = self.entropy[m] if entropy is None else entropy[m]
            high = x.max()
            log_q = x - use
            self.log_q[m] = log_q
            e = np.exp(log_q)
            # relative error of S: of its terms, weighted, and of their sum
            off_s = U * (4 + adds + 4 * (e * (high - x)).sum())
            off_x = 4 * U * (high - x)
            # ln S is at most ln V; logf and the last operations 4u of theirs
            self.off_log_q = off = off_s + off_x + 4 * U * (np.log(V) + (high - x))
            if lse is not None:  # log q = z·c − lse·log2(e), both to 48 bits; their difference and rounded sums
                off = 8 * U * (np.abs(log_q) + 2)
            t = int(at[m])
            has = 0 <= t < V
            if has:
                self.lim_logp[m] = (off_s + off_x + 4 * U * (np.log(V) + (high - x)))[t]
            self.lim_lse[m] = off_s + 4 * U * (np.log(V) + 2 * abs(high) + 1)
            # W/S: as S, each term by its x besides
            mean_x = (e * (high - x)).sum()
            self.lim_entropy[m] = lim_e = off_s * (1 + mean_x) + U * (
                (8 + adds) * mean_x + 8 * (e * (high - x) ** 2).sum() + 8 * np.log(V) + 4)
            gm, hm = abs(g[m]) if g is not None and has else 0.0, abs(h[m]) if h is not None else 0.0
            if entropy is not None:
                lim_e = 0.0
            d = e * (off + 8 * U) * (gm + hm * (np.abs(log_q) + ent)) + e * hm * (off + lim_e + 4 * U * (np.abs(log_q) + ent))
            d += 8 * U * e * (gm + hm * (np.abs(log_q) + ent))
            if has:
                d[t] += 4 * U * gm
            self.lim_dZ[m, :V] = d / tau + 4 * U * np.abs(self.dZ[m, :V])


def check(got, want, lim, kind, what):
    got = numpy(got)
    far = np.abs(got - want) - lim - HALF[kind] * (np.abs(want) + lim) - TINY[kind]
    far = np.where(got == want, -1.0, far)  # (equal infinities)
    assert not np.isnan(got).any(), f"{what}: NaN"
    at = np.unravel_index(np.argmax(far), far.shape)
    assert far[at] <= 0, f"{what}: {got[at]} for {want[at]} at {at}, {far[at]:.3e} past its bound"


def check_top(out, Z, tau, V, k, b):
    want = ref.top(numpy(Z), k, V)
    np.testing.assert_array_equal(out["top_index"].cpu().numpy(), want)
    got = numpy(out["top_logp"])
    for m in range(len(want)):
        n = (want[m] >= 0).sum()
        assert (got[m, n:] == -np.inf).all()
        at = want[m, :n]
        x = numpy(Z)[m, :V] / tau
        x = np.maximum(x, x.max() - 1e4)
        e = np.exp(b.log_q[m])
        lim = U * (4 + V / 64 + 64 + 4 * (e * (x.max() - x)).sum()) + 8 * U * (np.log(V) + x.max() - x[at])
        assert (np.abs(got[m, :n] - b.log_q[m, at]) <= lim + U * np.abs(b.log_q[m, at])).all()
        assert (np.diff(got[m, :n]) <= 0).all()


SHAPES = [
    # M, V, ldz, z, tau, k
    (1, 1, 1, "f32", 1.0, 1),
    (1, 7, 7, "bf16", 1.0, 9),
    (3, 8, 8, "f16", 2.0, 3),
    (2, 63, 64, "bf16", 0.5, 64),
    (5, 257, 264, "f32", 1.5, 20),
    (4, 1000, 1000, "bf16", 4.0, 256),
    (3, 1001, 1001, "f16", 1.0, 5),
    (3, 1003, 1003, "f32", 0.7, 50),
    (2, 2048, 2048, "f32", 1.0, 256),
    (2, 4104, 4104, "bf16", 1.0, 40),
    (3, 8200, 8203, "f16", 1.0, 17),
    (2, 16001, 16001, "f32", 1.0, 64),
    (3, 32003, 32008, "bf16", 1.0, 20),
    (2, 32768, 32768, "f32", 2.0, 33),
    (2, 40001, 40001, "f16", 1.0, 100),
    (2, 65500, 65528, "bf16", 1.0, 64),
    (2, 50001, 50008, "f32", 0.8, 256),
    (2, 131072, 131072, "bf16", 1.0, 50),
    (2, 128001, 128003, "f16", 1.0, 1),
]


@pytest.mark.parametrize("M,V,ld,z,tau,k", SHAPES)
def test_forward(M, V, ld, z, tau, k):
    print(f"logprobs forward {M} x {V} of {ld} {z} tau={tau} k={k}", flush=True)
    Z, target, g, h = rows(M, V, ld, z)
    b = Bounds(Z, target, tau, V, g, h)
    out = forward(Z, target, tau, V, k, g, h)
    check(out["logp"], b.logp, b.lim_logp, "f32", "logp")
    check(out["lse"], b.lse, b.lim_lse, "f32", "lse")
    check(out["entropy"], b.entropy, b.lim_entropy, "f32", "entropy")
    check(out["dZ"], b.dZ, b.lim_dZ, z, "dZ")
    check_top(out, Z, tau, V, k, b)
    # each result is the same to the bit without the others
    import torch as t
    alone = forward(Z, target, tau, V, stats=False)
    assert t.equal(alone["logp"], out["logp"])
    assert t.equal(forward(Z, target, tau, V, k)["top_logp"], out["top_logp"])
    likelihood = forward(Z, target, tau, V, 0, g, None)
    bg = Bounds(Z, target, tau, V, g)
    check(likelihood["dZ"], bg.dZ, bg.lim_dZ, z, "dZ of the likelihood")
    assert t.equal(forward(Z, target, tau, V, k, g, h, in_place=True)["dZ"], out["dZ"])
    # the given token among the top has the same log-probability
    same = out["top_index"] == target.cuda()[:, None]
    assert t.equal(out["top_logp"][same], out["logp"][same.any(1)])


@pytest.mark.parametrize("M,V,ld,z,tau,k", SHAPES)
def test_backward(M, V, ld, z, tau, k):
    import torch as t
    print(f"logprobs backward {M} x {V} of {ld} {z} tau={tau}", flush=True)
    Z, target, g, h = rows(M, V, ld, z, seed=1)
    out = forward(Z, target, tau, V)
    lse, entropy = out["lse"].cpu(), out["entropy"].cpu()
    for dl, de in ((g, None), (None, h), (g, h)):
        b = Bounds(Z, target, tau, V, dl, de, lse, entropy)
        got = backward(Z, target, tau, V, lse, entropy, dl, de)
        check(got, b.dZ, b.lim_dZ, z, "dZ")
        assert t.equal(backward(Z, target, tau, V, lse, entropy, dl, de, in_place=True), got)


@pytest.mark.parametrize("z", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [300, 9000, 20011, 50000, 140000])
@pytest.mark.parametrize("kind", ["equal", "two values", "rising", "few columns", "coarse"])
def test_top_of_unusual_rows(z, V, kind):
    """Rows where many columns reach the bound: the order is by logit, then by index."""
    import torch as t
    print(f"top of {kind} {V} {z}", flush=True)
    r = t.Generator().manual_seed(V)
    if kind == "equal":
        Z = t.full((2, V), 1.5)
        Z[1] = -2.25
    elif kind == "two values":
        Z = (t.rand(2, V, generator=r) < 0.5).float()
        Z[1] = t.where(t.rand(V, generator=r) < 20 / V, 1.0, -1.0)
    elif kind == "rising":
        Z = t.linspace(-20, 20, V).repeat(2, 1)
        Z[1] = Z[1].flip(0)
    elif kind == "few columns":
        Z = t.full((2, V), -float("inf"))
        Z[0, [5, V - 1, 77]] = t.tensor([1.0, 1.0, 2.0])
        Z[1] = -3e38 if z != "f16" else -float("inf")
        Z[1, 200:212] = 0.5
    else:
        Z = t.randn(2, V, generator=r).mul(2).round()
    Z, target = Z.to(types()[z]), t.tensor([5, 201], dtype=t.int32)
    for k in (1, 20, 256):
        out = forward(Z, target, 1.0, V, k)
        b = Bounds(Z, target, 1.0, V)
        check_top(out, Z, 1.0, V, k, b)
        check(out["entropy"], b.entropy, b.lim_entropy, "f32", "entropy")


@pytest.mark.parametrize("z", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [300, 9000, 50000, 140000])
@pytest.mark.parametrize("finite", [130, 200, 255])
def test_fewer_alternatives_than_asked_for_side_by_side(z, V, finite):
    """More columns next to one another than one wave lists, and still fewer than k."""
    import torch as t
    Z = t.full((2, V), -float("inf"))
    Z[0, 17:17 + finite] = t.randn(finite, generator=t.Generator().manual_seed(V)).mul(2).round()
    Z[1, V - finite:] = 0.5
    if z != "f16":
        Z[1, :8] = -1e30
    Z, target = Z.to(types()[z]), t.tensor([20, V - 1], dtype=t.int32)
    out = forward(Z, target, 1.0, V, 256)
    check_top(out, Z, 1.0, V, 256, Bounds(Z, target, 1.0, V))
    assert (out["top_index"][:, finite:] == -1).all()


@pytest.mark.parametrize("z,V", [("bf16", 700), ("f32", 2000), ("f16", 33000), ("bf16", 70001)])
def test_tokens_that_say_nothing(z, V):
    """No target, no gradient, masked rows: zeros, and untouched neighbours."""
    import torch as t
    Z, target, g, h = rows(8, V, V, z, seed=3)
    target[0] = -100
    target[1] = V
    g[2] = h[2] = 0.0
    Z[2, 3] = float("nan")
    Z[3] = -float("inf")
    Z[4] = -float("inf") if z == "f16" else -3.3e38
    Z[5, ::2] = -float("inf")
    target[5] = 1
    target[6] = -(2 ** 31)
    h[6] = 0.0
    out = forward(Z, target, 1.0, V, 4, g, h)
    got = {n: numpy(v) for n, v in out.items()}
    assert got["logp"][0] == 0 and got["logp"][1] == 0 and got["logp"][6] == 0
    assert not got["dZ"][[2, 3, 4, 6]].any()
    assert (got["logp"][3:5] == 0).all() and (got["entropy"][3:5] == 0).all() and (got["lse"][3:5] == -np.inf).all()
    assert (got["top_index"][3:5] == -1).all() and (got["top_logp"][3:5] == -np.inf).all()
    fine = [0, 1, 5, 6, 7]
    b = Bounds(Z[fine], target[fine], 1.0, V, g[fine], h[fine])
    check(out["dZ"][fine], b.dZ, b.lim_dZ, z, "dZ")
    check(out["entropy"][fine], b.entropy, b.lim_entropy, "f32", "entropy")
    lse, entropy = out["lse"].cpu(), out["entropy"].cpu()
    back = backward(Z, target, 1.0, V, lse, entropy, g, h)
    assert not numpy(back)[[2, 3, 4, 6]].any()
    b = Bounds(Z[fine], target[fine], 1.0, V, g[fine], h[fine], lse[fine], entropy[fine])
    check(back[fine], b.dZ, b.lim_dZ, z, "dZ from the saved sums")


@pytest.mark.parametrize("z,V", [("bf16", 700), ("f32", 2000), ("f16", 33000), ("bf16", 70001)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_a_number(z, V, value):
    import torch as t
    Z, target, g, h = rows(4, V, V, z, seed=4)
    Z[1, V // 3] = value
    Z[2] = -float("inf")
    Z[2, V - 1] = value
    target[1], target[2] = 0, -1
    out = forward(Z, target, 1.0, V, 4, g, h)
    lse, entropy = out["lse"], out["entropy"]
    back = backward(Z, target, 1.0, V, lse.cpu(), entropy.cpu(), g, h)
    for x in (lse, entropy):
        assert np.isnan(numpy(x)).tolist() == [False, True, True, False]
    assert np.isnan(numpy(out["logp"])).tolist() == [False, True, False, False]
    for x in (out["dZ"], back):
        assert np.isnan(numpy(x)[1:3]).all() and np.isfinite(numpy(x)[[0, 3]]).all()
    if np.isnan(value):
        clean = Z.clone()
        clean[1:3] = t.nan_to_num(clean[1:3].float(), nan=-float("inf"), neginf=-float("inf")).to(Z.dtype)
        np.testing.assert_array_equal(out["top_index"].cpu().numpy(), ref.top(numpy(clean), 4, V))


def test_padding_is_not_read_and_written_as_zeros():
    import torch as t
    Z, target, g, h = rows(5, 1003, 1031, "bf16", seed=5)
    other = Z.clone()
    other[:, 1003:] = float("nan")
    a, b = forward(Z, target, 1.0, 1003, 9, g, h), forward(other, target, 1.0, 1003, 9, g, h)
    for n in a:
        assert t.equal(a[n], b[n]), n
    assert not a["dZ"][:, 1003:].any()
    lse, entropy = a["lse"].cpu(), a["entropy"].cpu()
    x, y = backward(Z, target, 1.0, 1003, lse, entropy, g, h), backward(other, target, 1.0, 1003, lse, entropy, g, h)
    assert t.equal(x, y) and not x[:, 1003:].any()


def test_large_logits_of_one_sign():
    """fp32 logits near 2^20 with differences of order one: the exponents see the differences."""
    import torch as t
    Z, target, g, h = rows(3, 5000, 5000, "f32", seed=6)
    Z[0] += 2.0 ** 20
    Z[1] -= 2.0 ** 20
    out = forward(Z, target, 1.0, 5000, 8, g, h)
    # (tau = 1: c is log2(e) rounded, the same factor for z and its maximum; their
    # difference in x then carries an fma's rounding, 2^-24 of the difference)
    b = Bounds(Z, target, 1.0, 5000, g, h)
    check(out["logp"], b.logp, b.lim_logp, "f32", "logp")
    check(out["lse"], b.lse, b.lim_lse, "f32", "lse")
    check(out["entropy"], b.entropy, b.lim_entropy, "f32", "entropy")
    check(out["dZ"], b.dZ, b.lim_dZ, "f32", "dZ")
    check_top(out, Z, 1.0, 5000, 8, b)


def test_the_top_feeds_distillation():
    """A teacher's alternatives, as given, are the entries of the distillation loss; with itself it is near zero."""
    import torch as t
    Z, target, _, _ = rows(16, 4000, 4000, "f32", seed=7)
    teacher = forward(Z, target, 1.0, 4000, 64)
    loss, dZ = nan(16), nan(16, 4000)
    q.qlora_distill_fwd(Z.cuda(), teacher["top_logp"], teacher["top_index"], 1.0, None, loss, None, dZ)
    # log q of the entries over their own share: the loss is -log of the mass the top holds (64 terms of a few u
    # each, together below 64·32·u = 1.2e-4)
    mass = teacher["top_logp"].double().exp().sum(1)
    assert (loss.double() + mass.log()).abs().max() < 64 * 32 * U
