"""What is not a number in the layer with dropout and in the gated block: a dropped
one reaches no low-rank factor and no gradient of the adapters, and any other exactly
the outputs whose formulas hold it; all others keep their bits."""

import numpy as np
import pytest

from oracle import block as ref
from tests import gpu_util as G
from tests.test_gpu_adapters import within
from tests.test_gpu_block import Case

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def put(c, name, at, value):
    """`value` into an input, on the device and for the oracle."""
    c.dev[name][at] = value
    c.host[name] = c.dev[name].double().cpu().numpy()


@pytest.mark.parametrize("M", [4, 40, 65, 130, 300, 700])
@pytest.mark.parametrize("r", [8, 32, 64, 136])
@pytest.mark.parametrize("layers", [1, 2])
def test_dropped_values_reach_no_factor(M, r, layers):
    """Every dropped element of X is NaN or infinite.  (The base products, which see X
    itself, are NaN; the factors and the adapters' gradients are the oracle's.)"""
    import torch as t
    print(f"dropped NaN M={M} r={r} layers={layers}", flush=True)
    c = Case(M, 136, 320, r, layers, 0.3, seed=40)
    lost = t.from_numpy(c.mask == 0)
    bad = t.where(t.arange(lost.numel()).view_as(lost) % 3 > 0, NAN, INF).to(t.bfloat16)
    c.dev["X"].copy_(t.where(lost, bad, c.dev["X"].cpu()))
    c.host["X"] = c.dev["X"].double().cpu().numpy()
    T = c.linear(t.float32)[1][None] if layers == 1 else c.gated()[3]
    d = [c.host["dY"]] if layers == 1 else ref.gate_gradients(c.act, c.host["G"], c.host["U"], c.host["dY"])
    for saved in (T, None):
        if layers == 1:
            dX, *out = c.linear_backward(t.float32, None if saved is None else saved[0])
        else:
            dX, out = c.gated_backward(t.float32, saved)
        want_dX = size_dX = 0.0
        for l in range(layers):
            with np.errstate(invalid="ignore"):
                want_T, size_T = (c.forward_of(l, a)[1] for a in (False, True))
            within(T[l], want_T, size_T, c.K, f"T {l}")
            host_T = None if saved is None else saved[l].double().cpu().numpy()
            want, size = (c.backward_of(l, d[l], host_T, a) for a in (False, True))
            within(out[2 * l], want[1], size[1], c.N + 3 * M, f"dA {l}")
            within(out[2 * l + 1], want[2], size[2], c.K + 3 * M, f"dB {l}")
            want_dX, size_dX = want_dX + want[0], size_dX + size[0]
        within(dX, want_dX, size_dX, 2 * layers * (c.N + 2 * r), "dX")


def same(got, clean, finite, what):
    """Finite exactly where the oracle is, and there the bits of the run without the value."""
    import torch as t
    finite = t.from_numpy(np.ascontiguousarray(finite)).cuda()
    assert t.equal(t.isfinite(got), finite), what
    assert t.equal(t.where(finite, got, 0), t.where(finite, clean, 0)), what


@pytest.mark.parametrize("M", [3, 16, 40, 64, 130, 600])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_forward_of_tokens_that_are_not_numbers(M, value, act):
    import torch as t
    print(f"gated forward, {value} in X, M={M} {act}", flush=True)
    c = Case(M, 136, 320, 16, 2, 0.2, act, seed=41)
    clean = c.gated()
    bad = [0, M // 2]
    kept = np.argwhere(c.mask[bad[1]] != 0)[0, 0]
    put(c, "X", (bad[0], 17), value)
    put(c, "X", (bad[1], int(kept)), value)
    rows = np.ones(M, bool)
    rows[bad] = False
    got = c.gated()
    for x, y, what in zip(got[:3], clean[:3], "HGU"):
        same(x, y, np.repeat(rows[:, None], c.N, 1), what)
    for l in range(2):
        factor = rows.copy()
        factor[bad[0]] = c.mask[bad[0], 17] == 0 and bad[0] != bad[1]
        same(got[3][l], clean[3][l], np.repeat(factor[:, None], c.r, 1), "T")


@pytest.mark.parametrize("M", [3, 16, 40, 64, 130, 600])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["G", "U", "dY", "X", "dropped X"])
def test_backward_of_values_that_are_not_numbers(M, value, where):
    import torch as t
    print(f"gated backward, {value} in {where}, M={M}", flush=True)
    c = Case(M, 136, 320, 16, 2, 0.2, seed=42)
    m, n = M // 2, 33
    if where == "G" and value == INF:
        put(c, "G", (m, n), 1e38)   # (act' is 1 there as in the limit, so dG is a number, and the same one)
    clean = c.gated_backward(t.float32, None)
    if "X" in where:
        n = int(np.argwhere((c.mask[m] == 0) == (where == "dropped X"))[0, 0])
    put(c, where.split()[-1], (m, n), value)
    got = c.gated_backward(t.float32, None)
    with np.errstate(invalid="ignore", over="ignore"):
        d = ref.gate_gradients(c.act, c.host["G"], c.host["U"], c.host["dY"])
        want = [c.backward_of(l, d[l]) for l in range(2)]
    same(got[0], clean[0], np.isfinite(want[0][0]) & np.isfinite(want[1][0]), "dX")
    for l in range(2):
        same(got[1][2 * l], clean[1][2 * l], np.isfinite(want[l][1]), f"dA {l}")
        same(got[1][2 * l + 1], clean[1][2 * l + 1], np.isfinite(want[l][2]), f"dB {l}")
