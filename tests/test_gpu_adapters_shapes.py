"""The many-adapter layer at the sizes where its kernels change: every shape of
the dequant-GEMV (and several row groups per workgroup), both few-token forms
with and without split reductions, both GEMM tiles with and without, gradients
of one and of several units.  Bounds as in test_gpu_adapters; the weight is
dequantized on the device (bit-exact by its own tests)."""

import numpy as np
import pytest

from tests import gpu_util as G
from tests import test_gpu_adapters as A

pytestmark = pytest.mark.gpu


class Case(A.Case):
    """A.Case without the oracle's quantizer, for larger weights."""

    def __init__(self, *args, **kw):
        keep = G.oracle_quantized, G.oracle_w_hat
        try:
            G.oracle_quantized = lambda W: None
            G.oracle_w_hat = lambda q: np.zeros(args[1] * args[2], np.uint16)
            super().__init__(*args, **kw)
        finally:
            G.oracle_quantized, G.oracle_w_hat = keep
        self.W = G.bf16_f64(G.host_bf16(G.gpu_dequantize(self.w)))


SINGLE = [
    # M, N, K, r, count, kind            X in LDS, waves, row groups per workgroup
    (1, 4360, 512, 16, 3, "one"),        # 1 KB, 4 waves
    (1, 16648, 128, 8, 2, "one"),        # 4 waves, two groups for some
    (4, 4360, 2112, 40, 4, "each"),      # 17 KB, 8 waves
    (5, 8328, 1088, 16, 3, "mixed"),     # 8 waves, two groups for some
    (16, 4360, 2112, 64, 16, "each"),    # 68 KB, 16 waves, two groups for some
    (16, 264, 4416, 24, 5, "mixed"),     # 141 KB: X from memory
    (9, 136, 8256, 256, 3, "mixed"),     # X from memory, a long adapter row
    (3, 4104, 64, 8, 2, "mixed"),        # one block per row
]
MANY = [
    (20, 8328, 1856, 24, 9, "mixed"),    # 16 waves, 32 positions
    (50, 8328, 1856, 16, 30, "mixed"),   # 16 waves, 64 positions
    (40, 264, 2112, 32, 5, "each"),      # 8 waves, split
    (60, 2056, 2112, 64, 40, "mixed"),   # many adapters' stages shared by the splits
    (64, 136, 320, 256, 64, "each"),     # every token its own adapter, long ones
    (33, 520, 1088, 8, 2, "runs"),
    (100, 2056, 2112, 40, 7, "runs"),    # 256-row tiles, split
    (256, 1032, 1088, 16, 100, "each"),  # a hundred adapters in one tile
    (800, 264, 2112, 16, 5, "runs"),     # 512-row tiles, split
    (2048, 8328, 128, 8, 4, "runs"),     # 512-row tiles, direct
    (1600, 136, 8320, 16, 3, "mixed"),   # dX direct
    (1500, 264, 448, 16, 1, "one"),      # gradients of many units
    (2100, 72, 128, 24, 2, "runs"),      # units cut from long runs
]


@pytest.mark.parametrize("M,N,K,r,count,kind", SINGLE)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_few_tokens(M, N, K, r, count, kind, out):
    import torch as t
    print(f"adapters forward {M} x {N} x {K} r={r} count={count} {kind} {out}", flush=True)
    A.check_forward(Case(M, N, K, r, count, kind), t.bfloat16 if out == "bf16" else t.float32)


@pytest.mark.parametrize("M,N,K,r,count,kind", MANY)
@pytest.mark.parametrize("out,saved", [("bf16", True), ("f32", False)])
def test_many_tokens(M, N, K, r, count, kind, out, saved):
    import torch as t
    print(f"adapters both passes {M} x {N} x {K} r={r} count={count} {kind} {out}", flush=True)
    dtype = t.bfloat16 if out == "bf16" else t.float32
    c = Case(M, N, K, r, count, kind)
    _, T = A.check_forward(c, dtype)
    A.check_backward(c, dtype, T if saved else None)


@pytest.mark.parametrize("M,N,K,r,count,kind", [
    (7, 264, 320, 16, 3, "each"),
    (24, 264, 320, 8, 3, "each"),       # a split rank block of 16 and 16 zeros
    (32, 8328, 1856, 24, 4, "mixed"),
    (61, 264, 320, 24, 7, "each"),
    (64, 520, 1088, 64, 5, "runs"),
    (200, 264, 320, 16, 5, "each"),
    (300, 520, 1088, 40, 3, "runs"),
    (1100, 136, 320, 16, 6, "runs"),
])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_an_adapters_infinities_stay_its_tokens_own(M, N, K, r, count, kind, out):
    """One adapter's factors hold NaN and infinities: every token of another
    one, or of none, has the same bits as without them, and so have the other
    adapters' gradients."""
    import torch as t
    print(f"adapters with infinities {M} x {N} x {K} r={r} count={count} {kind} {out}", flush=True)
    dtype = t.bfloat16 if out == "bf16" else t.float32
    c = Case(M, N, K, r, count, kind)
    bad = int(c.index[M // 2]) if 0 <= c.index[M // 2] < count else 1
    own = t.from_numpy(np.flatnonzero(c.index == bad)).cuda()
    rest = t.from_numpy(np.flatnonzero(c.index != bad)).cuda()
    others = [a for a in range(count) if a != bad]
    Y, T = c.forward(dtype)
    want = c.backward(dtype, T)
    c.A[bad, r - 1, 3:9], c.B[bad, 5, :] = float("inf"), float("nan")
    c.B[bad, N - 1, 0], c.A[bad, :, K - 1] = float("-inf"), float("nan")
    bad_Y, bad_T = c.forward(dtype)
    got = c.backward(dtype, bad_T)
    assert t.equal(bad_Y[rest], Y[rest]) and t.equal(bad_T[rest], T[rest]) and t.equal(got[0][rest], want[0][rest])
    for a in others:
        assert t.equal(got[1][a], want[1][a]) and t.equal(got[2][a], want[2][a])
    assert len(own) == 0 or (bad_Y[own].isnan().any(1).all() and got[0][own].isnan().any(1).all())
