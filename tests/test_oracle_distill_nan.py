"""The distillation oracle where an input is not a number: NaN in that row's
results and in no other's, except where the row says nothing at all."""

import math

import numpy as np
import pytest

from oracle import distill


def rows():
    g = np.random.default_rng(2)
    Z, T = g.standard_normal((4, 9)), g.standard_normal((4, 3))
    return Z, T, np.stack([g.permutation(7)[:3] for _ in range(4)])


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_logit(value):
    Z, T, at = rows()
    Z[1, 4] = value
    with np.errstate(invalid="ignore"):
        loss, lse, dZ = distill.distill(Z, T, at, 2.0, vocab=7)
        _, _, saved = distill.distill(Z, T, at, 2.0, vocab=7, lse=lse)
    np.testing.assert_array_equal(np.isnan(loss), [False, True, False, False])
    np.testing.assert_array_equal(np.isnan(lse), np.isnan(loss))
    for d in (dZ, saved):
        assert np.isnan(d[1, :7]).all() and not d[:, 7:].any() and np.isfinite(d[[0, 2, 3]]).all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("entries", [1, 3])
def test_a_teachers_logit(value, entries):
    Z, T, at = rows()
    T[1, :entries] = value
    T[2, 0], at[2, 0] = value, -1  # no entry
    T[3, 1:], T[3, 0] = -math.inf, value
    with np.errstate(invalid="ignore"):
        loss, lse, dZ = distill.distill(Z, T, at, 2.0)
    np.testing.assert_array_equal(np.isnan(loss), [False, True, False, True])
    assert np.isfinite(lse).all()
    want = np.zeros((4, 9), bool)
    want[1, at[1]], want[3, at[3, 0]] = True, True
    np.testing.assert_array_equal(np.isnan(dZ), want)


def test_a_row_of_no_weight():
    Z, T, at = rows()
    Z[0], T[1] = math.nan, math.nan
    loss, _, dZ = distill.distill(Z, T, at, 1.0, weight=[0.0, 0.0, 1.0, 1.0])
    assert not loss[:2].any() and not dZ[:2].any() and (loss[2:] > 0).all()
