"""What is not a number in the distillation loss stays visible: a NaN or an
infinity among a row's logits, its saved log-sum-exp or its teacher's logits
gives NaN where the fp64 oracle has it, and nothing elsewhere; other rows stay
within the bounds of test_gpu_distill."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import distill as ref
from tests import test_gpu_distill as D

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# one chunk a thread, eight, 1,024 threads, and rows read twice (running sums); each with padding
LENGTHS = {"bf16": (1001, 1008), "f16": (32003, 32008), "f32": (32003, 32008), "bf16 long": (131077, 131080),
           "f32 long": (40001, 40004)}


def draw(form, k=12, seed=5, M=8):
    V, ld = LENGTHS[form]
    z = form.split()[0]
    Z, T, at, w = D.rows(M, V, ld, k, z, "f32", seed=seed)
    return Z, T, at, w, V, z


def backward(Z, T, at, tau, lse, w, V, in_place=False):
    import torch as t
    d = [x.cuda() for x in (Z, T, at, w)]
    dZ = d[0] if in_place else t.full_like(d[0], 7.0)
    q.qlora_distill_bwd(d[0], d[1], d[2], tau, lse, d[3], dZ, vocab=V)
    return dZ


def agree(got, want, clean, limits, kind, what):
    """NaN exactly where the oracle has it; the clean rows within their bounds."""
    nan = np.isnan(got.double().cpu().numpy())
    np.testing.assert_array_equal(nan, np.isnan(want), err_msg=what)
    D.check(got[clean], want[clean], limits, kind, what)


def both_passes(Z, T, at, w, V, z, bad, tau=1.25, backward_too=True):
    with np.errstate(invalid="ignore", divide="ignore"):
        want = ref.distill(Z.double().numpy(), T.double().numpy(), at.numpy(), tau, w.double().numpy(), V)
    clean = [m for m in range(len(Z)) if m not in bad]
    _, lim = D.bounds(Z[clean], T[clean], at[clean], tau, w[clean], V)
    got = D.call(Z, T, at, tau, w, V)
    for g, x, limit, kind, what in zip(got, want, lim, ("f32", "f32", z), ("loss", "lse", "dZ")):
        agree(g, x, clean, limit, kind, what)
    alone = D.call(Z, T, at, tau, w, V, part="loss")
    np.testing.assert_array_equal(alone[0].cpu().numpy(), got[0].cpu().numpy())
    np.testing.assert_array_equal(alone[1].cpu().numpy(), got[1].cpu().numpy())
    if not backward_too:
        return
    lse = got[1].cpu().numpy()
    with np.errstate(invalid="ignore", divide="ignore"):
        _, _, dz = ref.distill(Z.double().numpy(), T.double().numpy(), at.numpy(), tau, w.double().numpy(), V, lse)
    (_, _, _), lim = D.bounds(Z[clean], T[clean], at[clean], tau, w[clean], V, lse[clean])
    for in_place in (False, True):
        agree(backward(Z, T, at, tau, got[1], w, V, in_place), dz, clean, lim[2], z, "dZ from lse")


@pytest.mark.parametrize("form", LENGTHS)
def test_padding_is_zero_beside_a_row_that_is_not_a_number(form):
    import torch as t
    Z, T, at, w, V, z = draw(form)
    print(f"distill padding {form}", flush=True)
    Z[2, 17] = NAN
    Z[5, V - 1] = INF
    both_passes(Z, T, at, w, V, z, (2, 5), backward_too=False)
    lse = t.zeros(8, device="cuda")
    lse[3] = INF
    for in_place in (False, True):
        dZ = backward(Z, T, at, 1.25, lse, w, V, in_place)
        assert not dZ[:, V:].any()


@pytest.mark.parametrize("form", LENGTHS)
def test_gradient_from_a_saved_lse_that_is_not_a_number(form):
    Z, T, at, w, V, z = draw(form)
    print(f"distill saved lse {form}", flush=True)
    Z[1, V // 2] = NAN
    Z[3, 5] = INF
    Z[6, 0], Z[6, V - 1] = INF, NAN
    both_passes(Z, T, at, w, V, z, (1, 3, 6))


@pytest.mark.parametrize("form", LENGTHS)
def test_nan_columns_beside_a_finite_lse(form):
    """A log-sum-exp that is a number, of another pass over the logits: the NaN
    columns alone are NaN."""
    Z, T, at, w, V, z = draw(form)
    print(f"distill NaN columns {form}", flush=True)
    lse = D.call(Z, T, at, 1.25, w, V)[1]
    Z[2, 17], Z[4, V - 1], Z[6, V // 2:] = NAN, NAN, NAN
    with np.errstate(invalid="ignore"):
        _, _, want = ref.distill(Z.double().numpy(), T.double().numpy(), at.numpy(), 1.25, w.double().numpy(), V,
                                 lse.cpu().numpy())
    for in_place in (False, True):
        got = backward(Z, T, at, 1.25, lse, w, V, in_place).cpu()
        np.testing.assert_array_equal(got.isnan().numpy(), np.isnan(want))


@pytest.mark.parametrize("form", [f for f in LENGTHS if "long" not in f])
def test_a_row_of_nan_alone_is_not_a_masked_row(form):
    import torch as t
    Z, T, at, w, V, z = draw(form)
    print(f"distill rows of NaN {form}", flush=True)
    Z[0] = NAN
    Z[2] = -INF                            # masked
    Z[4] = -INF
    Z[4, V // 3] = NAN                     # masked but for a NaN
    Z[6] = t.finfo(Z.dtype).min if z != "f16" else -INF
    Z[6, 1] = NAN
    w[7] = 0.0                             # of no weight: nothing whatever it holds
    Z[7] = NAN
    got = D.call(Z, T, at, 1.25, w, V)
    assert got[0][7] == 0 and not got[2][7].any() and got[1][7].isnan()
    both_passes(Z[:7], T[:7], at[:7], w[:7], V, z, (0, 4, 6))


@pytest.mark.parametrize("form", [f for f in LENGTHS if "long" in f])
def test_nan_stretches_of_long_rows_reach_the_sum(form):
    """In rows that are read for a running maximum and sum: whole rows, one
    column, the chunks that a thread meets first or last, or all of its."""
    Z, T, at, w, V, z = draw(form)
    print(f"distill NaN stretches {form}", flush=True)
    per = 4 if z == "f32" else 8           # columns of a 16-byte chunk
    Z[0] = NAN
    Z[1, :per] = NAN
    Z[2, :2 * 1024 * per] = NAN            # every thread's first two chunks
    Z[3, V - 4 * per:] = NAN
    Z[4] = -INF                            # masked but for a NaN
    Z[4, V // 3] = NAN
    Z[5, :] = -INF                         # masked
    Z[6, :V - 9] = -INF                    # nine columns left
    both_passes(Z, T, at, w, V, z, (0, 1, 2, 3, 4))


@pytest.mark.parametrize("form", LENGTHS)
def test_teacher_logits_that_are_not_numbers(form):
    Z, T, at, w, V, z = draw(form)
    print(f"distill teacher {form}", flush=True)
    T[0, 3] = NAN
    T[1] = NAN
    T[2, 0] = INF
    T[3] = -INF                            # no entries
    T[4, 1:] = -INF
    T[4, 0] = NAN
    T[5, 2], at[5, 2] = NAN, -1            # no entry, whatever its logit is
    T[6], w[6] = NAN, 0.0
    both_passes(Z, T, at, w, V, z, (0, 1, 2, 4, 6))
    got = D.call(Z, T, at, 1.25, w, V)
    assert got[0][6] == 0 and not got[2][6].any()


@pytest.mark.parametrize("form", ["bf16", "f32 long"])
@pytest.mark.parametrize("tau", [0.25, 0.01])
def test_teacher_logits_whose_quotient_by_tau_passes_fp32(form, tau):
    """Their differences count: equal logits of any size are a uniform teacher,
    the far ones of a row with both have p = 0."""
    import torch as t
    Z, T, at, w, V, z = draw(form, M=4)
    print(f"distill large teacher {form} tau={tau}", flush=True)
    high, low = t.finfo(t.float32).max, t.finfo(t.float32).min
    T[0], T[1] = low, high
    T[2, ::2], T[2, 1::2] = high, low
    both_passes(Z, T, at, w, V, z, (), tau=tau)
    same = T.clone()
    same[:2] = 0.0
    same[2, ::2], same[2, 1::2] = 0.0, -INF
    got, want = D.call(Z, T, at, tau, w, V), D.call(Z, same, at, tau, w, V)
    assert all(t.equal(a, b) for a, b in zip(got, want))
