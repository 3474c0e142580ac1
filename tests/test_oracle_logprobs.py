"""The log-probability oracle against closed forms, brute force and differences."""

import math

import numpy as np
import pytest

from oracle import distill, logprobs


def test_closed_forms():
    Z = np.zeros((2, 8))
    logp, lse, ent, _ = logprobs.logprobs(Z, [3, -100], 1.0, vocab=5)
    np.testing.assert_allclose(logp, [-math.log(5), 0.0], rtol=1e-15)
    np.testing.assert_allclose(lse, [math.log(5)] * 2, rtol=1e-15)
    np.testing.assert_allclose(ent, [math.log(5)] * 2, rtol=1e-15)
    # two columns, one of them twice as likely
    logp, lse, ent, _ = logprobs.logprobs([[math.log(2.0) * 3, 0.0]], [0], 3.0)
    np.testing.assert_allclose([logp[0], lse[0]], [math.log(2 / 3), math.log(3)], rtol=1e-14)
    np.testing.assert_allclose(ent[0], math.log(3) - 2 / 3 * math.log(2), rtol=1e-14)
    # one column alone, and one left by the mask
    for z in ([[4.0]], [[4.0, -math.inf]], [[-math.inf, 4.0, -math.inf]]):
        t = int(np.argmax(z[0]))
        logp, lse, ent, dZ = logprobs.logprobs(z, [t], 1.0, g=[1.0], h=[1.0])
        assert (logp[0], lse[0], ent[0]) == (0.0, 4.0, 0.0) and not dZ.any()


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_the_gradient_is_the_difference(tau):
    g = np.random.default_rng(0)
    Z, target = g.standard_normal((4, 11)) * 2, np.array([2, 8, -1, 10])
    Z[1, 3] = -math.inf
    dl, de = g.standard_normal(4), g.standard_normal(4)

    def value(Z):
        logp, _, ent, _ = logprobs.logprobs(Z, target, tau, vocab=9)
        return (dl * logp + de * ent).sum()

    dZ = logprobs.logprobs(Z, target, tau, 9, dl, de)[3]
    step = 1e-6
    for m in range(4):
        for v in range(11):
            if not np.isfinite(Z[m, v]):
                assert dZ[m, v] == 0
                continue
            up, down = Z.copy(), Z.copy()
            up[m, v] += step
            down[m, v] -= step
            assert abs((value(up) - value(down)) / (2 * step) - dZ[m, v]) < 1e-8


def test_one_entry_of_distillation_is_the_likelihood():
    """A teacher with a single entry has p = 1 there: its loss is −logp and its gradient the likelihood's."""
    g = np.random.default_rng(1)
    Z, target = g.standard_normal((6, 20)), g.integers(0, 20, 6)
    loss, lse, dZ = distill.distill(Z, g.standard_normal((6, 1)), target[:, None], 1.0)
    logp, own, _, own_dZ = logprobs.logprobs(Z, target, 1.0, g=-np.ones(6))
    np.testing.assert_allclose(loss, -logp, rtol=1e-13)
    np.testing.assert_allclose(lse, own, rtol=1e-15)
    np.testing.assert_allclose(dZ, own_dZ, rtol=1e-12, atol=1e-16)


def test_rows_that_say_nothing_and_nan():
    Z = np.zeros((4, 6))
    Z[0] = -math.inf
    Z[1] = -3e38
    Z[2, 2] = math.nan
    Z[3, 2] = math.inf
    with np.errstate(invalid="ignore"):
        logp, lse, ent, dZ = logprobs.logprobs(Z, [0, 1, 2, -1], 1.0, g=np.ones(4), h=np.ones(4))
    assert (logp[:2] == 0).all() and (lse[:2] == -math.inf).all() and (ent[:2] == 0).all() and not dZ[:2].any()
    assert np.isnan(logp[2]) and logp[3] == 0 and np.isnan(lse[2:]).all() and np.isnan(ent[2:]).all()
    assert np.isnan(dZ[2:]).all()


def test_top():
    Z = np.array([[1.0, 3.0, 3.0, -math.inf, 2.0, 9.0], [0.0, -0.0, 0.0, math.nan, -1e31, 9.0]])
    np.testing.assert_array_equal(logprobs.top(Z, 5, vocab=5), [[1, 2, 4, 0, -1], [0, 1, 2, -1, -1]])
