"""Pins of the fp64 references for many adapters and for distillation: one
adapter reduces to the single-adapter layer, gradients agree with central
differences, and the loss has its closed-form values."""

import math

import numpy as np
import pytest

from oracle import adapters, distill, linalg


def problem(seed=0, M=7, N=6, K=5, r=3, count=3):
    g = np.random.default_rng(seed)
    return (g.standard_normal((M, K)), g.standard_normal((N, K)), g.standard_normal((count, r, K)),
            g.standard_normal((count, N, r)), g.uniform(0.5, 2, count), np.array([0, 2, -1, 2, 0, 5, 2])[:M],
            g.standard_normal((M, N)))


def test_one_adapter_is_the_single_adapter_layer():
    X, W, A, B, s, _, dY = problem()
    index = np.full(len(X), 1)
    Y, T = adapters.forward(X, W, A, B, s, index)
    Y1, T1 = linalg.linear_fwd(X, W, A[1], B[1], s[1] * 3, 3)
    np.testing.assert_allclose(Y, Y1, rtol=1e-12)
    np.testing.assert_allclose(T, T1, rtol=1e-12)
    got = adapters.backward(X, dY, W, A, B, s, index)
    want = linalg.linear_bwd(X, dY, W, A[1], B[1], s[1] * 3, 3)
    np.testing.assert_allclose(got[0], want[0], rtol=1e-11)
    np.testing.assert_allclose(got[1][1], want[1], rtol=1e-11)
    np.testing.assert_allclose(got[2][1], want[2], rtol=1e-11)
    assert not got[1][[0, 2]].any() and not got[2][[0, 2]].any()


def test_a_token_without_an_adapter_takes_the_base_alone():
    X, W, A, B, s, index, _ = problem()
    Y, T = adapters.forward(X, W, A, B, s, index)
    for m in (2, 5):  # -1 and past the pool
        np.testing.assert_allclose(Y[m], X[m] @ W.T, rtol=1e-12)
        assert not T[m].any()


@pytest.mark.parametrize("which", ["X", "A", "B"])
def test_gradients_agree_with_differences(which):
    X, W, A, B, s, index, dY = problem(3)
    dX, dA, dB = adapters.backward(X, dY, W, A, B, s, index)
    grad = {"X": dX, "A": dA, "B": dB}[which]
    v = {"X": X, "A": A, "B": B}[which]
    h = 1e-5
    for at in np.ndindex(v.shape):
        keep = v[at]
        f = []
        for step in (h, -h):
            v[at] = keep + step
            f.append((adapters.forward(X, W, A, B, s, index)[0] * dY).sum())
        v[at] = keep
        assert abs((f[0] - f[1]) / (2 * h) - grad[at]) < 1e-6 * (1 + abs(grad[at]))


def rows(seed=0, M=5, V=9, k=4):
    g = np.random.default_rng(seed)
    Z = g.standard_normal((M, V + 2)) * 2
    at = np.stack([g.permutation(V)[:k] for _ in range(M)])
    return Z, g.standard_normal((M, k)), at, g.uniform(0.5, 2, M), V


def test_loss_is_zero_where_the_student_answers_as_the_teacher():
    g = np.random.default_rng(1)
    t = g.standard_normal((3, 6))
    at = np.tile(np.arange(6), (3, 1))
    loss, lse, dZ = distill.distill(t + 4.0, t, at, 2.0)
    np.testing.assert_allclose(loss, 0, atol=1e-14)
    np.testing.assert_allclose(dZ, 0, atol=1e-14)


def test_one_entry_is_the_cross_entropy_of_its_column():
    Z, _, at, w, V = rows()
    loss, lse, dZ = distill.distill(Z, np.zeros((5, 1)), at[:, :1], 1.0, w, V)
    for m in range(5):
        q = np.exp(Z[m, :V]) / np.exp(Z[m, :V]).sum()
        assert math.isclose(loss[m], -w[m] * math.log(q[at[m, 0]]), rel_tol=1e-12)
        assert math.isclose(lse[m], math.log(np.exp(Z[m, :V]).sum()), rel_tol=1e-12)
    np.testing.assert_allclose(dZ.sum(1), 0, atol=1e-12)
    assert not dZ[:, V:].any()


@pytest.mark.parametrize("twice", [False, True])
def test_distillation_gradient_agrees_with_differences(twice):
    Z, t, at, w, V = rows(4)
    if twice:
        at[:, 1] = at[:, 0]
    at[1, 2] = -1
    at[2, 3] = V
    _, _, dZ = distill.distill(Z, t, at, 1.7, w, V)
    h = 1e-5
    for m, v in np.ndindex(Z.shape):
        keep = Z[m, v]
        f = []
        for step in (h, -h):
            Z[m, v] = keep + step
            f.append(distill.distill(Z, t, at, 1.7, w, V)[0].sum())
        Z[m, v] = keep
        assert abs((f[0] - f[1]) / (2 * h) - dZ[m, v]) < 1e-8


def test_rows_that_say_nothing():
    Z, t, at, w, V = rows(5)
    at[0] = -1
    t[1] = -np.inf
    w[2] = 0
    Z[3] = -np.inf
    loss, lse, dZ = distill.distill(Z, t, at, 1.0, w, V)
    assert not loss[:4].any() and not dZ[:4].any() and loss[4] > 0
    assert lse[3] == -math.inf and np.isfinite(lse[[0, 1, 2, 4]]).all()
