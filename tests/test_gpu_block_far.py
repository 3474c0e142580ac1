"""The gated block where its numbers are far apart: gate gradients whose factors are
tiny and huge, activations down to the smallest numbers."""

import numpy as np
import pytest

from oracle import block as ref
from tests import gpu_util as G
from tests.test_gpu_block import Case

pytestmark = pytest.mark.gpu


def bf16_of(x):
    import torch as t
    return t.from_numpy(np.asarray(x, dtype=np.float32)).to(t.bfloat16)


def spread(g, shape, low, high):
    """Values of either sign whose size is uniform in its logarithm."""
    return g.choice([-1.0, 1.0], shape) * 10.0 ** g.uniform(low, high, shape)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("kind", ["small dH", "smaller dH", "subnormal dH", "zero dH", "any size", "every g"])
def test_gate_gradients_of_far_factors(act, kind):
    """With T one-hot and s = 1 a column of dB is a token's dG or dU itself, to the
    bit.  (What overflows bf16 is left out by dH = 0 there: every other element is
    compared.)"""
    import torch as t
    print(f"gate gradients {act} {kind}", flush=True)
    M = r = 256
    N = 512
    shape = (M, N)
    c = Case(M, N, 64, r, 2, None, act, seed=7, alpha=float(r))
    g = np.random.default_rng(21)
    deep = g.uniform(-79, -20, shape) if act == "silu" else g.uniform(-9.7, -4, shape)
    value = {"small dH": (deep, spread(g, shape, 4, 30), spread(g, shape, -12, -4)),
             "smaller dH": (deep, spread(g, shape, 4, 30), spread(g, shape, -36, -12)),
             "subnormal dH": (np.where(g.random(shape) < 0.5, deep, g.standard_normal(shape)), spread(g, shape, 0, 38),
                              spread(g, shape, -40, -37)),
             "zero dH": (deep, spread(g, shape, 4, 38), np.where(g.random(shape) < 0.5, 0.0, spread(g, shape, -38, -30))),
             "any size": [spread(g, shape, -37, 37) for _ in range(3)],
             "every g": (g.standard_normal(shape), spread(g, shape, -3, 3), spread(g, shape, -3, 3))}[kind]
    for n, x in zip(("G", "U", "dY"), value):
        c.dev[n] = bf16_of(x).cuda()
    if kind == "every g":
        bits = np.arange(2 ** 17, dtype=np.int64).astype(np.uint16)
        c.dev["G"] = G.dev_bf16(np.where((bits & 0x7F80) == 0x7F80, 0x3F80, bits).astype(np.uint16).reshape(shape))
    host = [c.dev[n].double().cpu().numpy() for n in ("G", "U", "dY")]
    with np.errstate(over="ignore"):
        want = ref.gate_gradients(act, *host)
    lost = ~(np.isfinite(want[0]) & np.isfinite(want[1]))
    assert lost.mean() < 0.2
    c.dev["dY"][t.from_numpy(lost).cuda()] = 0.0
    T = t.eye(M, device="cuda").repeat(2, 1, 1)
    _, got = c.gated_backward(t.bfloat16, T)
    for l in range(2):
        x, y = got[2 * l + 1].double().cpu().numpy().T, np.where(lost, 0.0, want[l])
        assert np.isfinite(x).all()
        # (the products of MFMA flush what is below 2^-126)
        big = np.abs(y) >= 2.0 ** -126
        np.testing.assert_array_equal(x[big], y[big])
        assert (np.abs(x[~big]) < 2.0 ** -125).all()


@pytest.mark.parametrize("M", [1, 11, 40, 130, 700])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_the_activation_down_to_the_smallest_numbers(M, act):
    """G and U are picked from X one by one (zero weights, one-hot A), so H is
    act(g)·u alone: act within the error of its exponent, (6 + 2|h|)u for SiLU and
    (6 + 7|h|)u for GELU, and a step of fp32's subnormal numbers, which U scales."""
    import torch as t
    print(f"activation of far G, M={M} {act}", flush=True)
    N, K, r = 64, 128, 8
    c = Case(M, N, K, r, 2, None, act, seed=8, alpha=float(r))
    g = np.random.default_rng(31 + M)
    c.w = [G.gpu_quantize(G.dev_f32(np.zeros((N, K), np.float32))) for _ in range(2)]
    # row n of B takes rank n % 8, whose row of A takes element n % 8 (G) or 8 + n % 8 (U) of X
    for l in range(2):
        A = t.zeros(r, K, dtype=t.bfloat16)
        A[t.arange(r), 8 * l + t.arange(r)] = 1.0
        c.dev[f"A{l}"].copy_(A)
        c.dev[f"B{l}"].copy_(t.eye(r).repeat(N // r, 1))
    X = np.zeros((M, K))
    low = -104.0 if act == "silu" else -11.0
    X[:, :4] = g.uniform(low, 0.75 * low, (M, 4))
    X[:, 4:6] = g.uniform(low, -low, (M, 2))
    X[:, 6], X[:, 7] = spread(g, M, 2, 38), spread(g, M, -38, 0)
    X[:, 8:16] = spread(g, (M, 8), 0, 38)
    c.dev["X"].copy_(bf16_of(X))
    x = c.dev["X"].double().cpu().numpy()
    gv, uv = (np.tile(x[:, 8 * l:8 * l + 8], (1, N // r)) for l in range(2))
    value, _ = ref.act(act, gv)
    lost = ~np.isfinite(ref.bf16(value * uv))
    assert lost.mean() < 0.2
    h = np.abs(gv if act == "silu" else 1.5957691216057308 * (gv + 0.044715 * gv ** 3))
    u = 2.0 ** -24
    off = (6 + (2 if act == "silu" else 7) * np.minimum(h, 200) + 4) * u
    got = c.gated(save=False)[0].double().cpu().numpy()
    want = value * uv
    lim = off * np.abs(want) + 2.0 ** -149 * np.abs(uv)
    far = np.abs(got - want) - lim - 2.0 ** -8 * (np.abs(want) + lim) - 2.0 ** -126
    far = np.where(lost, -1.0, far)
    at = np.unravel_index(np.argmax(far), far.shape)
    assert not np.isnan(got).any() and far[at] <= 0, f"H {got[at]} for {want[at]}, g={gv[at]}, u={uv[at]}"
