"""The dropout and gated-block oracle: the generator against its published test
vectors, the mask's share and independence, formulas against differences."""

import numpy as np
import pytest

from oracle import block


@pytest.mark.parametrize("counter,key,expect", [
    # known answers of the 4x32, 10-round generator
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((block.LOW,) * 4, (block.LOW,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator(counter, key, expect):
    assert tuple(block.philox4x32(counter, key)) == expect


def test_pieces_are_the_generators():
    seed, offset = 0x0123456789ABCDEF, 0xFEDCBA9876543210
    got = block.pieces(3, 24, seed, offset).reshape(-1)
    for i in range(72):
        words = block.philox4x32((i // 8, 0, offset & block.LOW, offset >> 32), (seed & block.LOW, seed >> 32))
        assert got[i] == (words[i % 8 // 2] >> (16 * (i % 2))) & 0xFFFF


@pytest.mark.parametrize("p", [0.0, 2.0 ** -16, 0.05, 0.1, 0.5, 0.99])
def test_share_and_mean(p):
    """n elements of a share within five deviations; the mean of keep is 1 within as many."""
    M, K = 512, 640
    k = block.keep(M, K, p, 7, 3)
    t = round(65536 * p) / 65536
    dev = np.sqrt(t * (1 - t) / (M * K))
    assert abs((k == 0).mean() - t) <= 5 * dev
    assert abs(k.mean() - 1) <= 5 * dev / (1 - t)


def test_other_seeds_and_offsets_are_other_masks():
    base = block.keep(64, 64, 0.5, 1, 0) != 0
    for seed, offset in ((2, 0), (1 << 32 | 1, 0), (1, 1), (1, 1 << 32)):
        same = (base == (block.keep(64, 64, 0.5, seed, offset) != 0)).mean()
        assert abs(same - 0.5) < 5 * 0.5 / 64


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_activation_and_slope(kind):
    g = np.linspace(-12, 12, 481)
    value, slope = block.act(kind, g)
    up, down = block.act(kind, g + 1e-5)[0], block.act(kind, g - 1e-5)[0]
    np.testing.assert_allclose((up - down) / 2e-5, slope, atol=1e-9)
    ref = g * (0.5 + 0.5 * np.tanh(g / 2)) if kind == "silu" else \
        0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    np.testing.assert_allclose(value, ref, rtol=1e-9, atol=1e-14)
    far = block.act(kind, np.array([-1e30, -200.0, 200.0, 1e30]))
    np.testing.assert_allclose(far[0], [0, 0, 200, 1e30], atol=1e-80)
    np.testing.assert_allclose(far[1], [0, 0, 1, 1], atol=1e-80)


def test_rounding():
    np.testing.assert_array_equal(block.bf16([1.0, 1 + 2 ** -8, 1 + 3 * 2 ** -8, 1 + 2 ** -8 + 2 ** -20, -0.0, np.inf]),
                                  [1.0, 1.0, 1 + 2 ** -6, 1 + 2 ** -7, 0.0, np.inf])


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_the_gradients_are_the_differences(p):
    g = np.random.default_rng(0)
    M, N, K, r, s = 3, 8, 64, 8, 0.7
    X, W, A, B = (g.standard_normal(x) for x in ((M, K), (N, K), (r, K), (N, r)))
    dY, mask = g.standard_normal((M, N)), block.keep(M, K, p, 5)
    dX, dA, dB = block.backward(X, dY, W, A, B, s, mask)

    def value():
        return (dY * block.forward(X, W, A, B, s, mask)[0]).sum()

    for x, d in ((X, dX), (A, dA), (B, dB)):
        for at in [tuple(g.integers(0, n) for n in x.shape) for _ in range(20)]:
            old = x[at]
            x[at] = old + 1e-5
            up = value()
            x[at] = old - 1e-5
            down = value()
            x[at] = old
            assert abs((up - down) / 2e-5 - d[at]) < 1e-7 * max(1, abs(d[at]))


def test_a_dropped_nan_is_gone():
    X = np.ones((1, 64))
    mask = block.keep(1, 64, 0.5, 1)
    X[0, np.flatnonzero(mask[0] == 0)[0]] = np.nan
    A, B, W = np.ones((8, 64)), np.ones((8, 8)), np.zeros((8, 64))
    assert np.isfinite(block.forward(X, W, A, B, 1.0, mask)[1]).all()
