"""Distillation from a teacher's top logits against the fp64 oracle.  Bounds
per element, u = 2^-24: an exponential is off by 4u·(1 + |its exponent|) of
itself, the row's sum by the additions of one thread and of the reduction,
the output by half a step of its type."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import distill as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}


def types():
    import torch as t
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}


def rows(M, V, ld, k, z, top, seed=0, scale=3.0):
    import torch as t
    g = t.Generator().manual_seed(seed)
    Z = (t.randn(M, ld, generator=g) * scale).to(types()[z])
    at = t.stack([t.randperm(V, generator=g)[:k] if k <= V else t.randint(0, V, (k,), generator=g)
                  for _ in range(M)]).to(t.int32)
    T = (t.randn(M, k, generator=g) * scale).to(types()[top])
    w = t.rand(M, generator=g) + 0.25
    return Z, T, at, w


def call(Z, T, at, tau, w, V, part="both", in_place=False):
    import torch as t
    M = Z.shape[0]
    d = [None if x is None else x.cuda() for x in (Z, T, at, w)]
    loss, lse = t.full((M,), float("nan"), device="cuda"), t.full((M,), float("nan"), device="cuda")
    dZ = None if part == "loss" else d[0] if in_place else t.full(Z.shape, float("nan"), dtype=Z.dtype, device="cuda")
    q.qlora_distill_fwd(d[0], d[1], d[2], tau, d[3], loss, lse, dZ, vocab=V)
    return loss, lse, dZ


def bounds(Z, T, at, tau, w, V, given=None):
    """(loss, lse, dZ) in 64 bits and what each may be off by, before the output's rounding."""
    z, t, a = Z.double().numpy(), T.double().numpy(), at.numpy()
    wt = np.ones(len(z)) if w is None else w.double().numpy()
    loss, lse, dZ = ref.distill(z, t, a, tau, wt, V, given)
    M, k = t.shape
    lim_loss, lim_lse, lim_dz = np.zeros(M), np.zeros(M), np.zeros_like(z)
    adds = V / 64 + 64  # additions of one thread (at least 64 of them share a row) and of the reduction
    for m in range(M):
        use = lse[m] if given is None else float(given[m])
        if use == -np.inf:
            continue
        x = np.maximum(z[m, :V] / tau, -1e4)
        high = x.max()
        size = abs(high) + abs(use) + 4
        lim_lse[m] = U * (4 * size + adds + 4 * 16)
        ok = (a[m] >= 0) & (a[m] < V) & (t[m] > -np.inf)
        if not ok.any() or wt[m] == 0:
            continue
        y = np.maximum(t[m][ok] / tau, -1e4)
        y_range = y.max() - y.min()
        p = np.exp(y - y.max()) / np.exp(y - y.max()).sum()
        off_p = p * U * (16 + 8 * (y.max() - y) + k)
        log_p, log_q = y - y.max() - np.log(np.exp(y - y.max()).sum()), x[a[m][ok]] - use
        gap = np.abs(log_p - log_q)
        lim_loss[m] = abs(wt[m]) * tau ** 2 * (
            (p * (lim_lse[m] + U * (8 * (np.abs(log_p) + np.abs(log_q) + np.abs(x[a[m][ok]]) + np.abs(y) + size)
                                    + 8 * y_range + k))).sum()
            + (off_p * gap).sum() + U * (k + 8) * (p * gap).sum())
        e = np.exp(x - use)
        lim_dz[m, :V] = e * U * (32 + 8 * np.maximum(np.abs(x - use), high - x) + adds)
        np.add.at(lim_dz[m], a[m][ok], off_p + p * U * 4)
        lim_dz[m] *= abs(wt[m]) * tau
        lim_dz[m] += 4 * U * np.abs(dZ[m])
    return (loss, lse, dZ), (lim_loss, lim_lse, lim_dz)


def check(got, want, lim, kind, what):
    got = got.double().cpu().numpy()
    far = np.abs(got - want) - lim - HALF[kind] * (np.abs(want) + lim) - TINY[kind]
    far = np.where(got == want, -1.0, far)  # (equal infinities)
    assert not np.isnan(got).any(), f"{what}: NaN"
    at = np.unravel_index(np.argmax(far), far.shape)
    assert far[at] <= 0, f"{what}: {got[at]} for {want[at]} at {at}, {far[at]:.3e} past its bound"


def check_all(Z, T, at, tau, w, V, z):
    (loss, lse, dZ), lim = bounds(Z, T, at, tau, w, V)
    got = call(Z, T, at, tau, w, V)
    check(got[0], loss, lim[0], "f32", "loss")
    check(got[1], lse, lim[1], "f32", "lse")
    check(got[2], dZ, lim[2], z, "dZ")
    return got


SHAPES = [
    # M, V, ldz, k, z, top, tau
    (1, 1, 1, 1, "f32", "f32", 1.0),
    (1, 7, 7, 3, "bf16", "f32", 1.0),
    (3, 8, 8, 8, "f16", "f16", 2.0),
    (2, 63, 64, 5, "bf16", "bf16", 0.5),
    (5, 257, 264, 33, "f32", "bf16", 1.5),
    (4, 1000, 1000, 512, "bf16", "f16", 4.0),
    (3, 1001, 1001, 17, "f16", "f32", 1.0),
    (3, 1003, 1003, 17, "f32", "f16", 0.7),
    (2, 2048, 2048, 64, "f32", "f32", 1.0),
    (2, 4099, 4104, 256, "bf16", "f32", 2.0),
    (2, 8191, 8191, 2, "bf16", "f32", 1.0),
    (2, 16391, 16392, 20, "f32", "f32", 3.0),
    (2, 32003, 32003, 64, "bf16", "bf16", 1.0),
    (1, 50001, 50008, 50, "f16", "f32", 1.0),
    (1, 65543, 65543, 8, "f32", "f32", 1.0),
    (1, 131077, 131080, 100, "bf16", "f32", 2.0),
    (1, 300007, 300007, 30, "bf16", "f32", 1.0),
    (1, 270001, 270001, 30, "f32", "f32", 1.0),
]


@pytest.mark.parametrize("M,V,ld,k,z,top,tau", SHAPES)
def test_loss_and_gradient(M, V, ld, k, z, top, tau):
    import torch as t
    print(f"distill {M} x {V} ({ld}) k={k} {z} {top} tau={tau}", flush=True)
    Z, T, at, w = rows(M, V, ld, k, z, top)
    got = check_all(Z, T, at, tau, w, V, z)
    # the loss alone, in place, without weights, and the gradient from the saved lse
    alone = call(Z, T, at, tau, w, V, part="loss")
    assert t.equal(alone[0], got[0]) and t.equal(alone[1], got[1])
    assert t.equal(call(Z, T, at, tau, w, V, in_place=True)[2], got[2])
    d = [x.cuda() for x in (Z, T, at, w)]
    dZ = t.full_like(d[0], float("nan"))
    q.qlora_distill_bwd(d[0], d[1], d[2], tau, got[1], d[3], dZ, vocab=V)
    (_, _, want), lim = bounds(Z, T, at, tau, w, V, got[1].cpu().numpy())
    check(dZ, want, lim[2], z, "dZ from lse")
    z2 = d[0].clone()
    q.qlora_distill_bwd(z2, d[1], d[2], tau, got[1], d[3], z2, vocab=V)
    assert t.equal(z2, dZ)
    one = call(Z, T, at, tau, None, V)
    (loss, _, dz1), lim = bounds(Z, T, at, tau, None, V)
    check(one[0], loss, lim[0], "f32", "loss without weights")
    check(one[2], dz1, lim[2], z, "dZ without weights")


@pytest.mark.parametrize("z", ["f32", "bf16", "f16"])
def test_rows_that_say_nothing(z):
    """Rows without entries, of weight 0 with NaN logits, with every column
    masked, with a teacher of −infinity; masked columns; columns twice."""
    import torch as t
    V, k = 777, 40
    Z, T, at, w = rows(12, V, 784, k, z, "f32", seed=3)
    at[0] = -1
    at[1] = t.tensor([V, -1, 2 ** 31 - 1, -2 ** 31] * 10, dtype=t.int32)
    T[2] = -float("inf")
    w[3] = 0.0
    Z[4] = -float("inf")
    T[5, 3:] = -float("inf")               # three entries left
    at[6, 1::2] = at[6, 0::2]              # every column twice
    at[7] = 5                              # one column 40 times
    Z[8, ::3] = -float("inf")              # masked columns, none of them an entry
    at[8] = t.arange(k, dtype=t.int32) * 3 + 1
    Z[9, 1:] = t.finfo(types()[z]).min     # one column left, the rest at the type's lowest
    at[9] = 0
    T[10] = -3e38                          # entries at the lowest value are entries
    at[11, 1:] = -1
    (loss, lse, dZ), lim = bounds(Z, T, at, 1.25, w, V)
    Z[3, 100] = float("nan")
    got = call(Z, T, at, 1.25, w, V)
    keep = [m for m in range(12) if m != 3]
    check(got[0], loss, lim[0], "f32", "loss")
    check(got[1][keep], lse[keep], lim[1][keep], "f32", "lse")
    check(got[2], dZ, lim[2], z, "dZ")
    for m in (0, 1, 2, 3, 4):
        assert got[0][m] == 0 and not got[2][m].any()
    d = [x.cuda() for x in (Z, T, at, w)]
    got_b = t.full_like(d[0], float("nan"))
    saved = got[1].clone()
    saved[3] = 1.0
    q.qlora_distill_bwd(d[0], d[1], d[2], 1.25, saved, d[3], got_b, vocab=V)
    (_, _, want), lim = bounds(t.where(t.isnan(Z), 0, Z), T, at, 1.25, w, V, saved.cpu().numpy())
    check(got_b, want, lim[2], z, "dZ from lse")


def test_padding_columns_are_not_read_and_come_back_zero():
    import torch as t
    Z, T, at, w = rows(6, 50, 77, 9, "bf16", "f32")
    first = call(Z, T, at, 1.0, w, 50)
    Z[:, 50:] = float("nan")
    again = call(Z, T, at, 1.0, w, 50)
    assert all(t.equal(a, b) for a, b in zip(first, again))
    assert not again[2][:, 50:].any()


def test_rows_after_the_last_are_left_alone():
    import torch as t
    Z, T, at, w = rows(9, 301, 301, 5, "bf16", "f32")
    d = [x.cuda() for x in (Z, T, at, w)]
    dZ, loss = t.full_like(d[0], 7.0), t.full((9,), 7.0, device="cuda")
    q.qlora_distill_fwd(d[0][:8], d[1][:8], d[2][:8], 1.0, d[3][:8], loss[:8], None, dZ[:8])
    assert (dZ[8] == 7.0).all() and loss[8] == 7.0 and not (dZ[:8] == 7.0).any()


def test_gradient_agrees_with_differences():
    """Along one direction in fp32: the loss is smooth in z with second
    derivative at most w per unit step (tau² · 1/tau²), so the central
    difference over ±h is off by less than w·h²·|v|³ and by the loss's rounding
    over h."""
    import torch as t
    Z, T, at, w = rows(6, 400, 400, 24, "f32", "f32", seed=8, scale=1.5)
    tau, h = 1.5, 2.0 ** -6
    v = t.randn(6, 400, generator=t.Generator().manual_seed(3)) / 20  # |v| about 1 per row
    _, _, dZ = call(Z, T, at, tau, w, 400)
    up, down = (call(Z + s * h * v, T, at, tau, w, 400, part="loss")[0].double().cpu() for s in (1, -1))
    got = (up - down) / (2 * h)
    along = (dZ.double().cpu() * v.double()).sum(1)
    _, lim = bounds(Z, T, at, tau, w, 400)
    norm = v.double().norm(dim=1)
    # (Z ± h·v is rounded to fp32: the step is off by u·|z| per column, its effect by the gradient's size, at most 2·w·tau)
    bound = w.double() * h * h * norm ** 3 + t.from_numpy(lim[0]) / h + 2 * w.double() * tau * U * 8 / h
    assert ((got - along).abs() <= bound).all(), (got, along, bound)


def test_graph_replays():
    import torch as t
    Z, T, at, w = (x.cuda() for x in rows(33, 5003, 5008, 20, "bf16", "f32", seed=6))
    loss, lse, dZ, dB = t.empty(33, device="cuda"), t.empty(33, device="cuda"), t.empty_like(Z), t.empty_like(Z)

    def step():
        q.qlora_distill_fwd(Z, T, at, 2.0, w, loss, lse, dZ, vocab=5003)
        q.qlora_distill_bwd(Z, T, at, 2.0, lse, w, dB, vocab=5003)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    for rep in range(3):
        print(f"distill replay {rep}", flush=True)
        Z.copy_(t.randn(33, 5008, device="cuda") * 2)
        step()
        t.cuda.synchronize()
        want = [o.clone() for o in (loss, lse, dZ, dB)]
        for o in (loss, lse, dZ, dB):
            o.fill_(float("nan"))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip((loss, lse, dZ, dB), want))
