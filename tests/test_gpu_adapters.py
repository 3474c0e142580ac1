"""The linear layer of a batch whose tokens carry different adapters, against
the fp64 oracle: every element within the rounding bound of fp32 accumulation
(2u per addition, u = 2^-24, over the sums of absolute terms) plus half a step
of the output type."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import adapters as ref
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def assignment(kind, M, count, seed=0):
    g = np.random.default_rng(seed)
    if kind == "each":       # interleaved, every adapter in turn
        return (np.arange(M) % count).astype(np.int32)
    if kind == "mixed":      # any order, some tokens without one (any value outside the pool)
        a = g.integers(0, count, M)
        a[g.random(M) < 0.25] = g.choice([-1, count, -7, 2 ** 31 - 1, -2 ** 31])
        return a.astype(np.int32)
    if kind == "runs":       # one request after another, uneven lengths
        cuts = np.sort(g.integers(0, M + 1, count - 1))
        return np.repeat(g.permutation(count), np.diff(np.concatenate(([0], cuts, [M])))).astype(np.int32)
    if kind == "one":
        return np.full(M, count - 1, np.int32)
    assert kind == "none"
    return np.full(M, -1, np.int32)


class Case:
    def __init__(self, M, N, K, r, count, kind, seed=0):
        import torch as t
        g = np.random.default_rng(1000 + seed)
        self.M, self.N, self.K, self.r, self.count = M, N, K, r, count
        W = (g.standard_normal((N, K)) * 0.02).astype(np.float32)
        self.w = G.gpu_quantize(G.dev_f32(W))
        self.W = G.bf16_f64(G.oracle_w_hat(G.oracle_quantized(W))).reshape(N, K)

        def bf(*shape, scale=1.0):
            return t.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(t.bfloat16)

        self.X, self.dY = bf(M, K), bf(M, N)
        self.A, self.B = bf(count, r, K, scale=0.05), bf(count, N, r, scale=0.05)
        self.s = t.from_numpy(g.uniform(0.25, 4.0, count).astype(np.float32))
        self.index = assignment(kind, M, count, seed)
        self.host = tuple(x.double().numpy() for x in (self.X, self.dY, self.A, self.B, self.s))
        self.X, self.dY, self.A, self.B, self.s = (x.cuda() for x in (self.X, self.dY, self.A, self.B, self.s))
        self.pool = q.AdapterPool(self.A, self.B, self.s)
        self.plan = q.AdapterPlan.empty(M, count)
        self.plan.buffer.fill_(0xA5)
        q.qlora_adapters_plan(t.from_numpy(self.index).cuda(), self.plan)
        self.sizes = q.qlora_adapters_sizes(N, K, M, r, count)

    def scratch(self, key):
        import torch as t
        return t.full((max(256, self.sizes[key]),), 0xA5, dtype=t.uint8, device="cuda")

    def forward(self, dtype, save=True):
        import torch as t
        Y = t.full((self.M, self.N), float("nan"), dtype=dtype, device="cuda")
        T = t.full((self.M, self.r), float("nan"), device="cuda") if save else None
        q.qlora_adapters_fwd(self.w, self.X, self.pool, self.plan, Y, T, self.scratch("fwd_ws_bytes"))
        return Y, T

    def backward(self, dtype, T):
        import torch as t
        dX = t.full((self.M, self.K), float("nan"), dtype=dtype, device="cuda")
        dA = t.full((self.count, self.r, self.K), float("nan"), device="cuda")
        dB = t.full((self.count, self.N, self.r), float("nan"), device="cuda")
        q.qlora_adapters_bwd(self.w, self.X, self.dY, self.pool, self.plan, T, dX, dA, dB,
                             self.scratch("bwd_ws_bytes"))
        return dX, dA, dB


def within(got, want, size, terms, what, half_step=0.0):
    """|got - want| <= 2u·terms·size + half a step of the output, per element."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    far = np.abs(got - want) - (2 * U * (terms + 16) * size + half_step * (np.abs(want) + 2 * U * terms * size))
    at = np.unravel_index(np.argmax(far), far.shape) if far.size else None
    assert far.size == 0 or far[at] <= 0, f"{what}: {got[at]} for {want[at]} at {at}, {far[at]:.3e} past its bound"


def check_forward(c, dtype, save=True):
    import torch as t
    X, _, A, B, s = c.host
    Y, T = c.forward(dtype, save)
    want, want_T = ref.forward(X, c.W, A, B, s, c.index)
    size, size_T = ref.forward(X, c.W, A, B, s, c.index, absolute=True)
    # K additions of T and of the base, 3·r of the up-projection's three-part split
    within(Y, want, size, 2 * c.K + 4 * c.r, "Y", 2.0 ** -8 if dtype == t.bfloat16 else 0.0)
    if save:
        within(T, want_T, size_T, c.K, "T")
    return Y, T


def check_backward(c, dtype, T):
    import torch as t
    X, dY, A, B, s = c.host
    host_T = None if T is None else T.double().cpu().numpy()
    got = c.backward(dtype, T)
    want = ref.backward(X, dY, c.W, A, B, s, c.index, host_T)
    size = ref.backward(X, dY, c.W, A, B, s, c.index, host_T, absolute=True)
    within(got[0], want[0], size[0], 2 * c.N + 4 * c.r, "dX", 2.0 ** -8 if dtype == t.bfloat16 else 0.0)
    within(got[1], want[1], size[1], c.N + 3 * c.M, "dA")
    within(got[2], want[2], size[2], c.K + 3 * c.M, "dB")
    return got


SHAPES = [
    # M, N, K, r, count, tokens' adapters
    (1, 8, 64, 8, 1, "one"),
    (1, 264, 320, 16, 5, "one"),
    (1, 264, 320, 16, 5, "none"),
    (2, 24, 4160, 32, 3, "each"),
    (5, 520, 192, 64, 3, "mixed"),
    (16, 264, 704, 24, 40, "each"),
    (16, 136, 448, 256, 2, "mixed"),
    (17, 264, 320, 40, 17, "each"),
    (31, 8, 64, 8, 1024, "mixed"),
    (64, 512, 256, 64, 4, "runs"),
    (65, 328, 576, 16, 9, "mixed"),
    (130, 264, 320, 136, 7, "runs"),
    (200, 520, 128, 8, 300, "mixed"),
    (257, 264, 320, 72, 5, "runs"),
    (300, 776, 256, 32, 2, "mixed"),
    (513, 136, 832, 48, 33, "each"),
    (600, 264, 192, 128, 3, "one"),
    (700, 264, 192, 16, 6, "none"),
]


@pytest.mark.parametrize("M,N,K,r,count,kind", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_forward(M, N, K, r, count, kind, out):
    import torch as t
    print(f"adapters forward {M} x {N} x {K} r={r} count={count} {kind} {out}", flush=True)
    c = Case(M, N, K, r, count, kind)
    check_forward(c, t.bfloat16 if out == "bf16" else t.float32, save=out == "f32" or M % 2 == 0)


@pytest.mark.parametrize("M,N,K,r,count,kind", SHAPES)
@pytest.mark.parametrize("out,saved", [("bf16", False), ("f32", True)])
def test_backward(M, N, K, r, count, kind, out, saved):
    import torch as t
    print(f"adapters backward {M} x {N} x {K} r={r} count={count} {kind} {out} saved={saved}", flush=True)
    c = Case(M, N, K, r, count, kind, seed=1)
    T = c.forward(t.float32)[1] if saved else None
    check_backward(c, t.bfloat16 if out == "bf16" else t.float32, T)


def test_no_tokens():
    import torch as t
    c = Case(0, 264, 320, 16, 3, "one")
    c.forward(t.bfloat16)
    _, dA, dB = c.backward(t.bfloat16, None)
    assert not dA.any() and not dB.any()


def test_plan_sorts_the_tokens_stably():
    import torch as t
    for M, count, kind in ((1, 1, "one"), (63, 5, "mixed"), (1024, 1024, "mixed"), (5000, 77, "mixed"),
                           (4097, 3, "runs"), (300, 4, "none"), (2500, 1000, "each")):
        index = assignment(kind, M, count, seed=3)
        plan = q.AdapterPlan.empty(M, count)
        q.qlora_adapters_plan(t.from_numpy(index).cuda(), plan)
        words = plan.buffer.view(t.int32).cpu().numpy()
        pad = lambda n: -(-n // 16) * 16  # noqa: E731
        at = np.cumsum([0, 16, pad(M), pad(M), pad(M), pad(count + 1), pad(count + 1)])
        head, owner, perm, group, ids, start, slot = (words[a:] for a in at)
        clean = np.where((index >= 0) & (index < count), index, -1)
        key = np.where(clean < 0, count, clean)
        used = np.unique(clean[clean >= 0])
        assert head[0] == len(used) and head[1] == (clean >= 0).sum()
        np.testing.assert_array_equal(owner[:M], clean)
        np.testing.assert_array_equal(perm[:M], np.argsort(key, kind="stable"))
        np.testing.assert_array_equal(ids[:len(used)], used)
        np.testing.assert_array_equal(start[:len(used) + 1],
                                      np.concatenate((np.searchsorted(np.sort(key), used), [head[1]])))
        want = np.full(count, -1)
        want[used] = np.arange(len(used))
        np.testing.assert_array_equal(slot[:count], want)
        np.testing.assert_array_equal(group[:M], np.where(np.sort(key) < count, want[np.sort(key) % count], len(used)))


def test_adapters_without_tokens_are_not_read():
    import torch as t
    for M in (9, 150):
        c = Case(M, 264, 320, 16, 6, "mixed")
        keep = c.index[c.index == c.index.clip(0, 5)]
        idle = [a for a in range(6) if a not in keep[:4]]
        c.index = np.where(np.isin(c.index, idle), -1, c.index).astype(np.int32)
        q.qlora_adapters_plan(t.from_numpy(c.index).cuda(), c.plan)
        for a in idle:
            c.A[a], c.B[a], c.s[a] = float("nan"), float("inf"), float("nan")
        host = list(c.host)
        for i in (2, 3, 4):
            host[i] = host[i].copy()
            host[i][idle] = 0.0
        c.host = tuple(host)
        check_forward(c, t.float32)
        check_backward(c, t.float32, None)


def test_a_tokens_infinities_stay_its_own():
    import torch as t
    for M in (12, 200):
        c = Case(M, 264, 320, 16, 3, "each")
        bad = [1, 7]             # adapters 1 and 1: adapters 0 and 2 keep their gradients
        c.X[1, 3], c.dY[1, 5], c.X[7, 0] = float("inf"), float("nan"), float("nan")
        clean = Case(M, 264, 320, 16, 3, "each")
        rest = [m for m in range(M) if m not in bad]
        assert t.equal(c.forward(t.float32)[0][rest], clean.forward(t.float32)[0][rest])
        got, want = c.backward(t.float32, None), clean.backward(t.float32, None)
        assert t.equal(got[0][rest], want[0][rest])
        for a in (0, 2):
            assert t.equal(got[1][a], want[1][a]) and t.equal(got[2][a], want[2][a])


def test_equal_calls_give_equal_bits_in_any_order_of_rows():
    """Two runs agree bit for bit, and permuting the tokens permutes the rows
    of Y and dX to the same values."""
    import torch as t
    for M in (11, 300):
        c = Case(M, 264, 448, 32, 5, "mixed")
        first, again = c.forward(t.float32), c.forward(t.float32)
        assert t.equal(first[0], again[0]) and t.equal(first[1], again[1])
        g1, g2 = c.backward(t.float32, first[1]), c.backward(t.float32, first[1])
        assert all(t.equal(a, b) for a, b in zip(g1, g2))


def test_graph_replays_and_another_stream():
    """Plan, forward and backward captured into one graph with two layers that
    share a workspace; replays with other adapters and inputs in the same
    buffers, eager work in between."""
    import torch as t
    for M in (7, 150):
        c = Case(M, 264, 320, 16, 4, "runs")
        index = t.from_numpy(c.index).cuda()
        wsf, wsb = c.scratch("fwd_ws_bytes"), c.scratch("bwd_ws_bytes")
        Y, T = t.empty(M, 264, dtype=t.bfloat16, device="cuda"), t.empty(M, 16, device="cuda")
        dX = t.empty(M, 320, dtype=t.bfloat16, device="cuda")
        dA, dB = t.empty(4, 16, 320, device="cuda"), t.empty(4, 264, 16, device="cuda")
        outs = (Y, T, dX, dA, dB)

        def step():
            q.qlora_adapters_plan(index, c.plan)
            q.qlora_adapters_fwd(c.w, c.X, c.pool, c.plan, Y, T, wsf)
            q.qlora_adapters_bwd(c.w, c.X, c.dY, c.pool, c.plan, T, dX, dA, dB, wsb)

        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            step()
        t.cuda.current_stream().wait_stream(side)
        t.cuda.synchronize()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            step()
        g = t.Generator(device="cuda").manual_seed(5)
        for rep in range(3):
            print(f"adapters graph M={M} replay {rep}", flush=True)
            index.copy_(t.randint(-1, 4, (M,), generator=g, device="cuda", dtype=t.int32))
            c.X.copy_(t.randn(M, 320, generator=g, device="cuda"))
            step()
            t.cuda.synchronize()
            want = [o.clone() for o in outs]
            for o in outs:
                o.fill_(float("nan"))
            wsf.fill_(0xFF), wsb.fill_(0xFF), c.plan.buffer.fill_(0xFF)
            t.cuda.synchronize()
            graph.replay()
            t.cuda.synchronize()
            assert all(t.equal(a, b) for a, b in zip(outs, want))


def test_gradients_agree_with_differences():
    """d<Y, dY>/dθ by central differences of the layer itself in fp32, along
    one random direction for X, A and B each: Y is linear in X and bilinear in
    A and B, so the difference has no truncation error in any of them, and its
    rounding is 2u·(2K + 4r + 16) of the terms' absolute sum on either side."""
    import torch as t
    c = Case(70, 136, 192, 16, 3, "mixed", seed=2)
    dX, dA, dB = c.backward(t.float32, None)
    X, dY, A, B, s = c.host
    g = t.Generator().manual_seed(9)
    for name, grad in (("X", dX), ("A", dA), ("B", dB)):
        v = getattr(c, name)
        keep = v.clone()
        h = 2.0 ** -3
        step = (t.randint(0, 2, v.shape, generator=g) * 2 - 1).cuda()
        ends, terms = [], 0.0
        for sign in (1, -1):
            v.copy_((keep.float() + sign * h * step).bfloat16())
            moved = v.double().cpu().numpy()
            now = {"X": X, "A": A, "B": B, name: moved}
            terms += (ref.forward(now["X"], c.W, now["A"], now["B"], s, c.index, absolute=True)[0] * np.abs(dY)).sum()
            ends.append(((c.forward(t.float32)[0].double() * c.dY.double()).sum(), v.double()))
        v.copy_(keep)
        # (the steps are rounded to bf16 with the values: the direction taken is their difference.  A and B move
        # about `keep` unevenly by that rounding, which enters only through products of two moved factors: none here)
        along = float((grad.double() * (ends[0][1] - ends[1][1])).sum())
        got = float(ends[0][0] - ends[1][0])
        bound = 2 * U * (2 * c.K + 2 * c.N + 3 * c.M + 4 * c.r + 32) * terms
        assert abs(got - along) <= bound, (name, got, along, bound)
