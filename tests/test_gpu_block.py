"""The linear layer with dropout of its adapter's input, and the gated
feed-forward block, against the fp64 oracle: every element within the rounding
bound of fp32 accumulation (2u per addition, u = 2^-24, over the sums of absolute
terms) plus half a step of the output type; the mask and the gate's gradients to
the bit."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import block as ref
from tests import gpu_util as G
from tests.test_gpu_adapters import U, within

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
SEED, OFFSET = 0x1234567890ABCDEF, 0x0FEDCBA987654321


class Case:
    def __init__(self, M, N, K, r, layers, p, act="silu", seed=0, alpha=None):
        import torch as t
        g = np.random.default_rng(2000 + seed)
        self.M, self.N, self.K, self.r, self.layers, self.act = M, N, K, r, layers, act
        self.alpha = 2.0 * r if alpha is None else alpha
        self.s = self.alpha / r
        self.w, self.W = [], []
        for _ in range(layers):
            W = (g.standard_normal((N, K)) * 0.04).astype(np.float32)
            self.w.append(G.gpu_quantize(G.dev_f32(W)))
            self.W.append(G.bf16_f64(G.oracle_w_hat(G.oracle_quantized(W))).reshape(N, K))

        def bf(*shape, scale=1.0):
            return t.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(t.bfloat16)

        x = {"X": bf(M, K), "dY": bf(M, N), "G": bf(M, N, scale=2.0), "U": bf(M, N, scale=2.0)}
        x |= {f"A{l}": bf(r, K, scale=0.05) for l in range(layers)}
        x |= {f"B{l}": bf(N, r, scale=0.05) for l in range(layers)}
        self.host = {n: v.double().numpy() for n, v in x.items()}
        self.dev = {n: v.cuda() for n, v in x.items()}
        self.drop = q.Dropout(p, SEED, OFFSET) if p is not None else None
        self.mask = ref.keep(M, K, p or 0.0, SEED, OFFSET)
        self.sizes = (q.qlora_gated_sizes if layers == 2 else q.qlora_dropout_linear_sizes)(N, K, M, r)
        if layers == 2:
            self.adapters = q.GatedAdapters(*(self.dev[n] for n in ("A0", "B0", "A1", "B1")), self.alpha)

    def scratch(self, key):
        import torch as t
        return t.full((max(256, self.sizes[key]),), 0xFF, dtype=t.uint8, device="cuda")

    def nan(self, *shape, dtype=None):
        import torch as t
        return t.full(shape, float("nan"), dtype=dtype or t.float32, device="cuda")

    def linear(self, dtype, save=True):
        d, Y, T = self.dev, self.nan(self.M, self.N, dtype=dtype), self.nan(self.M, self.r) if save else None
        q.qlora_dropout_linear_fwd(self.w[0], d["X"], d["A0"], d["B0"], self.r, self.alpha, self.drop, Y, T,
                                   self.scratch("fwd_ws_bytes"))
        return Y, T

    def linear_backward(self, dtype, T):
        d = self.dev
        out = self.nan(self.M, self.K, dtype=dtype), self.nan(self.r, self.K), self.nan(self.N, self.r)
        q.qlora_dropout_linear_bwd(self.w[0], d["X"], d["dY"], d["A0"], d["B0"], self.r, self.alpha, self.drop, T, *out,
                                   self.scratch("bwd_ws_bytes"))
        return out

    def gated(self, save=True):
        import torch as t
        H = self.nan(self.M, self.N, dtype=t.bfloat16)
        Gs, Us = (self.nan(self.M, self.N, dtype=t.bfloat16) if save else None for _ in range(2))
        T = self.nan(2, self.M, self.r) if save else None
        q.qlora_gated_fwd(self.w[0], self.w[1], self.dev["X"], self.adapters, self.act, self.drop, H, Gs, Us, T,
                          self.scratch("fwd_ws_bytes"))
        return H, Gs, Us, T

    def gated_backward(self, dtype, T):
        d = self.dev
        dX = self.nan(self.M, self.K, dtype=dtype)
        out = [self.nan(*s) for s in ((self.r, self.K), (self.N, self.r)) * 2]
        q.qlora_gated_bwd(self.w[0], self.w[1], d["X"], d["dY"], d["G"], d["U"], self.adapters, self.act, self.drop, T,
                          dX, *out, self.scratch("bwd_ws_bytes"))
        return dX, out

    def forward_of(self, layer, absolute=False):
        h = self.host
        return ref.forward(h["X"], self.W[layer], h[f"A{layer}"], h[f"B{layer}"], self.s, self.mask, absolute)

    def backward_of(self, layer, dY, T=None, absolute=False):
        h = self.host
        return ref.backward(h["X"], dY, self.W[layer], h[f"A{layer}"], h[f"B{layer}"], self.s, self.mask, T, absolute)


def check_linear(c, dtype, save=True):
    import torch as t
    Y, T = c.linear(dtype, save)
    want, want_T = c.forward_of(0)
    size, size_T = c.forward_of(0, True)
    # K additions of T and of the base, 3·r of the up-projection's three-part split
    within(Y, want, size, 2 * c.K + 4 * c.r, "Y", HALF_BF16 if dtype == t.bfloat16 else 0.0)
    if save:
        within(T, want_T, size_T, c.K, "T")
    return Y, T


def check_linear_backward(c, dtype, T):
    import torch as t
    host_T = None if T is None else T.double().cpu().numpy()
    got = c.linear_backward(dtype, T)
    want, size = (c.backward_of(0, c.host["dY"], host_T, a) for a in (False, True))
    within(got[0], want[0], size[0], 2 * c.N + 4 * c.r, "dX", HALF_BF16 if dtype == t.bfloat16 else 0.0)
    within(got[1], want[1], size[1], c.N + 3 * c.M, "dA")
    within(got[2], want[2], size[2], c.K + 3 * c.M, "dB")
    return got


SHAPES = [
    # M, N, K, r, p
    (1, 8, 64, 8, 0.5),
    (1, 264, 320, 16, 0.1),
    (2, 24, 4160, 32, 0.05),
    (5, 520, 192, 64, None),
    (9, 4360, 704, 24, 0.3),
    (16, 264, 704, 24, 0.9),
    (16, 136, 448, 256, 0.1),
    (13, 72, 11008, 8, 0.2),
    (17, 264, 320, 40, 0.1),
    (31, 8, 64, 8, 0.5),
    (64, 512, 256, 64, 0.05),
    (65, 328, 576, 16, 0.1),
    (130, 264, 320, 136, 0.0),
    (200, 520, 128, 8, 0.999),
    (257, 264, 320, 72, 0.1),
    (300, 776, 256, 32, None),
    (513, 136, 832, 48, 0.25),
    (600, 264, 192, 128, 0.1),
    (2100, 1032, 192, 16, 0.05),
]


@pytest.mark.parametrize("M,N,K,r,p", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear(M, N, K, r, p, out):
    import torch as t
    print(f"dropout linear {M} x {N} x {K} r={r} p={p} {out}", flush=True)
    check_linear(Case(M, N, K, r, 1, p), t.bfloat16 if out == "bf16" else t.float32, save=out == "f32" or M % 2 == 0)


@pytest.mark.parametrize("M,N,K,r,p", SHAPES)
@pytest.mark.parametrize("out,saved", [("bf16", False), ("f32", True)])
def test_linear_backward(M, N, K, r, p, out, saved):
    import torch as t
    print(f"dropout linear backward {M} x {N} x {K} r={r} p={p} {out} saved={saved}", flush=True)
    c = Case(M, N, K, r, 1, p, seed=1)
    T = c.linear(t.bfloat16)[1] if saved else None
    got = check_linear_backward(c, t.bfloat16 if out == "bf16" else t.float32, T)
    again = c.linear_backward(got[0].dtype, T)
    assert all(t.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("M", [3, 20, 300])
@pytest.mark.parametrize("p", [2.0 ** -16, 0.1, 0.5, 65535 / 65536])
def test_mask_of_every_pass_to_the_bit(M, p):
    """With one-hot rows of A, T is D(X) itself; with a weight of zeros dX is the masked low-rank product alone, and
    dA from one-hot V picks tokens' D(X)."""
    import torch as t
    print(f"mask M={M} p={p}", flush=True)
    N, K, r = 256, 512, 256
    c = Case(M, N, K, r, 1, p, alpha=float(r))
    c.w[0] = G.gpu_quantize(G.dev_f32(np.zeros((N, K), np.float32)))
    X = c.host["X"]
    D = np.float32(1) * (X * c.mask)  # c·x: one product, rounded once where T is
    for half in range(2):
        A = t.zeros(r, K, dtype=t.bfloat16)
        A[t.arange(r), half * r + t.arange(r)] = 1.0
        c.dev["A0"].copy_(A)
        _, T = c.linear(t.float32)
        got = T.double().cpu().numpy()
        # (c in fp32, one rounding of the product)
        want = D[:, half * r:(half + 1) * r]
        assert ((got != 0) == (want != 0)).all()
        assert (np.abs(got - want) <= 2 * U * np.abs(want)).all()
    # dY·B = ones, A of ones: dX = r·keep
    c.dev["A0"].fill_(1.0)
    c.dev["B0"].copy_(t.eye(N))
    c.dev["dY"].fill_(1.0)
    dX, _, _ = c.linear_backward(t.float32, None)
    got = dX.double().cpu().numpy()
    assert ((got != 0) == (c.mask != 0)).all()
    # (a sum of r equal terms in three parts each: 3r additions of 2u, as everywhere here)
    assert np.abs(got - r * c.mask).max() <= 2 * U * (3 * r) * r * c.mask.max()
    # V one-hot: row m of dY is e_m
    c.dev["dY"].copy_(t.eye(N)[:M] if M <= N else t.eye(N).repeat(2, 1)[:M])
    _, dA, _ = c.linear_backward(t.bfloat16, None)
    want = np.zeros((r, K))
    for m in range(M):
        want[m % N] += (X * c.mask)[m]
    got = dA.double().cpu().numpy()
    size = np.zeros((r, K))
    for m in range(M):
        size[m % N] += np.abs(X * c.mask)[m]
    assert ((got == 0) >= (size == 0)).all()
    assert (np.abs(got - want) <= 6 * U * size).all()


def test_no_dropout_is_the_plain_layer():
    """p = 0 or None against qlora_linear_fwd and qlora_linear_bwd: the same sums, so within both bounds."""
    import torch as t
    c = Case(130, 264, 320, 16, 1, None, seed=2)
    Y, T = c.linear(t.float32)
    d = c.dev
    Y2, T2 = G.gpu_forward(c.w[0], d["X"], d["A0"], d["B0"], c.r, c.alpha, t.float32)
    _, size = c.forward_of(0), c.forward_of(0, True)
    assert (np.abs((Y - Y2).double().cpu().numpy()) <= 4 * U * (2 * c.K + 4 * c.r + 16) * size[0]).all()
    assert (np.abs((T - T2).double().cpu().numpy()) <= 4 * U * (c.K + 16) * size[1]).all()
    c.drop = q.Dropout(0.0, 1)
    assert t.equal(c.linear(t.float32)[0], Y)


def test_offset_on_the_device():
    """Dropout.step is added to the offset when the kernels run."""
    import torch as t
    for M in (5, 40):
        c = Case(M, 64, 128, 8, 1, 0.5, seed=3)
        step = t.tensor([7], dtype=t.int64, device="cuda")
        c.drop = q.Dropout(0.5, SEED, 2 ** 64 - 4, step)
        c.mask = ref.keep(M, 128, 0.5, SEED, 3)  # (2^64 - 4 + 7 passes 2^64)
        check_linear(c, t.bfloat16)
        check_linear_backward(c, t.bfloat16, None)
        step.fill_(2 ** 32 + 4)
        c.mask = ref.keep(M, 128, 0.5, SEED, 2 ** 32)
        check_linear(c, t.bfloat16)
        check_linear_backward(c, t.bfloat16, None)


@pytest.mark.parametrize("M", [4, 40])
def test_a_dropped_nan_reaches_no_factor(M):
    import torch as t
    c = Case(M, 64, 128, 8, 1, 0.5, seed=4)
    c.w[0] = G.gpu_quantize(G.dev_f32(np.zeros((64, 128), np.float32)))
    lost = t.from_numpy(c.mask == 0).cuda()
    c.dev["X"][lost] = float("nan")
    _, T = c.linear(t.float32)
    assert t.isfinite(T).all()
    dX, dA, dB = c.linear_backward(t.float32, T)
    assert all(t.isfinite(x).all() for x in (dX, dA, dB))


def check_gated(c, save=True):
    H, Gs, Us, T = c.gated(save)
    want, size = [c.forward_of(l) for l in range(2)], [c.forward_of(l, True) for l in range(2)]
    off = [2 * U * (2 * c.K + 4 * c.r + 16) * s[0] for s in size]
    value, _ = ref.act(c.act, want[0][0])
    # act is steep by less than 1.13; its own roundings and the product's below 16u
    lim = 1.13 * off[0] * (np.abs(want[1][0]) + off[1]) + np.abs(value) * off[1] + 16 * U * np.abs(value * want[1][0])
    got = H.double().cpu().numpy()
    far = np.abs(got - value * want[1][0]) - lim - HALF_BF16 * (np.abs(value * want[1][0]) + lim) - 2.0 ** -126
    assert np.isfinite(got).all() and (far <= 0).all(), f"H: {far.max():.3e} past its bound"
    if save:
        for l, x in enumerate((Gs, Us)):
            within(x, want[l][0], size[l][0], 2 * c.K + 4 * c.r, "GU"[l], HALF_BF16)
            within(T[l], want[l][1], size[l][1], c.K, "T")
    return H, Gs, Us, T


def check_gated_backward(c, dtype, T):
    import torch as t
    dX, got = c.gated_backward(dtype, T)
    d = ref.gate_gradients(c.act, c.host["G"], c.host["U"], c.host["dY"])
    want_dX, size_dX = 0.0, 0.0
    for l in range(2):
        host_T = None if T is None else T[l].double().cpu().numpy()
        want, size = (c.backward_of(l, d[l], host_T, a) for a in (False, True))
        want_dX, size_dX = want_dX + want[0], size_dX + size[0]
        within(got[2 * l], want[1], size[1], c.N + 3 * c.M, f"dA {l}")
        within(got[2 * l + 1], want[2], size[2], c.K + 3 * c.M, f"dB {l}")
    within(dX, want_dX, size_dX, 4 * c.N + 8 * c.r, "dX", HALF_BF16 if dtype == t.bfloat16 else 0.0)
    return dX, got


@pytest.mark.parametrize("M,N,K,r,p", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated(M, N, K, r, p, act):
    import torch as t
    print(f"gated {M} x {N} x {K} r={r} p={p} {act}", flush=True)
    c = Case(M, N, K, r, 2, p, act, seed=5)
    H = check_gated(c)[0]
    assert t.equal(c.gated(save=False)[0], H)


@pytest.mark.parametrize("M,N,K,r,p", SHAPES)
@pytest.mark.parametrize("act,out,saved", [("silu", "bf16", True), ("gelu_tanh", "f32", False)])
def test_gated_backward(M, N, K, r, p, act, out, saved):
    import torch as t
    print(f"gated backward {M} x {N} x {K} r={r} p={p} {act} {out} saved={saved}", flush=True)
    c = Case(M, N, K, r, 2, p, act, seed=6)
    T = c.gated()[3] if saved else None
    dX, got = check_gated_backward(c, t.bfloat16 if out == "bf16" else t.float32, T)
    dX2, again = c.gated_backward(dX.dtype, T)
    assert t.equal(dX, dX2) and all(t.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("kind", ["every g", "every g, small", "normal", "wide", "extreme"])
def test_gate_gradients_to_the_bit(act, kind):
    """With T one-hot and s = 1 a column of dB is a token's dG or dU itself."""
    import torch as t
    print(f"gate gradients {act} {kind}", flush=True)
    M = r = 256
    N = 512
    c = Case(M, N, 64, r, 2, None, act, seed=7, alpha=float(r))
    g = np.random.default_rng(8)
    if kind.startswith("every g"):  # all finite bf16 values (256·512 of them are twice as many as there are)
        bits = np.arange(2 ** 17, dtype=np.int64).astype(np.uint16)
        bits = np.where((bits & 0x7F80) == 0x7F80, 0x3F80, bits).astype(np.uint16).reshape(M, N)
        c.dev["G"] = G.dev_bf16(bits)
        if kind == "every g, small":  # so that nothing overflows
            for n in ("U", "dY"):
                c.dev[n] = t.from_numpy(g.uniform(-0.8, 0.8, (M, N)).astype(np.float32)).to(t.bfloat16).cuda()
    elif kind in ("wide", "extreme"):
        far = 11 if kind == "wide" else 30  # (three of 10^11 times a normal one do not overflow)
        for n in ("G", "U", "dY"):
            x = t.from_numpy(g.standard_normal((M, N)).astype(np.float32) * 10.0 ** g.uniform(-far, far, (M, N)).astype(np.float32))
            x[t.from_numpy(g.random((M, N)) < 0.1)] = 0.0
            c.dev[n] = x.to(t.bfloat16).cuda()
    T = t.eye(M, device="cuda").repeat(2, 1, 1)
    _, got = c.gated_backward(t.bfloat16, T)
    host = [c.dev[n].double().cpu().numpy() for n in ("G", "U", "dY")]
    want = ref.gate_gradients(act, *host)
    for l in range(2):
        x = got[2 * l + 1].double().cpu().numpy().T
        # (a value that overflows bf16 is an infinity, and a column with one is NaN beside it: 0·inf)
        fine = np.isfinite(want[l]).all(0)
        assert kind in ("every g", "extreme") or fine.all()
        # (the products of MFMA flush what is below 2^-126)
        big = (np.abs(want[l]) >= 2.0 ** -126) & fine
        np.testing.assert_array_equal(x[big], want[l][big])
        assert (np.abs(x[fine[None] & ~big]) < 2.0 ** -125).all()


def test_no_tokens():
    import torch as t
    for layers in (1, 2):
        c = Case(0, 64, 128, 8, layers, 0.1)
        if layers == 1:
            c.linear(t.bfloat16)
            out = c.linear_backward(t.bfloat16, None)[1:]
        else:
            c.gated()
            out = c.gated_backward(t.bfloat16, None)[1]
        assert not any(x.any() for x in out)


def test_full_size():
    """A 7B projection pair at 2,048 tokens: sampled rows and columns against the oracle."""
    import torch as t
    print("gated 2048 x 11008 x 4096", flush=True)
    M, N, K, r, p = 2048, 11008, 4096, 64, 0.1
    g = np.random.default_rng(9)
    dev = t.Generator("cuda").manual_seed(3)

    def bf(*shape, scale=1.0):
        return (t.randn(*shape, generator=dev, device="cuda") * scale).to(t.bfloat16)

    w = [G.gpu_quantize(t.randn(N, K, generator=dev, device="cuda") * 0.02) for _ in range(2)]
    W = [G.gpu_dequantize(x) for x in w]
    X, dH, Gv, Uv = bf(M, K), bf(M, N), bf(M, N, scale=1.3), bf(M, N, scale=1.3)
    A, B = [bf(r, K, scale=0.02) for _ in range(2)], [bf(N, r, scale=0.02) for _ in range(2)]
    ad, drop = q.GatedAdapters(A[0], B[0], A[1], B[1], 16.0), q.Dropout(p, 11, 12)
    size = q.qlora_gated_sizes(N, K, M, r)
    H, Gs, Us = (t.empty(M, N, dtype=t.bfloat16, device="cuda") for _ in range(3))
    T = t.empty(2, M, r, device="cuda")
    q.qlora_gated_fwd(w[0], w[1], X, ad, "silu", drop, H, Gs, Us, T, q.workspace(size["fwd_ws_bytes"]))
    mask = ref.keep(M, K, p, 11, 12)
    x, s = X.double().cpu().numpy(), 16.0 / r
    rows = np.sort(g.choice(M, 40, replace=False))
    for l, out in enumerate((Gs, Us)):
        a, b, wl = A[l].double().cpu().numpy(), B[l].double().cpu().numpy(), W[l].double().cpu().numpy()
        want, want_T = ref.forward(x[rows], wl, a, b, s, mask[rows])
        lim, lim_T = ref.forward(x[rows], wl, a, b, s, mask[rows], absolute=True)
        at = t.from_numpy(rows).cuda()
        within(out[at], want, lim, 2 * K + 4 * r, "GU"[l], HALF_BF16)
        within(T[l][at], want_T, lim_T, K, "T")
    dX = t.empty(M, K, dtype=t.float32, device="cuda")
    grads = [t.empty(*n, device="cuda") for n in ((r, K), (N, r)) * 2]
    q.qlora_gated_bwd(w[0], w[1], X, dH, Gv, Uv, ad, "silu", drop, T, dX, *grads, q.workspace(size["bwd_ws_bytes"]))
    d = ref.gate_gradients("silu", *(v.double().cpu().numpy() for v in (Gv, Uv, dH)))
    want_dX = lim_dX = 0.0
    for l in range(2):
        a, b, wl = A[l].double().cpu().numpy(), B[l].double().cpu().numpy(), W[l].double().cpu().numpy()
        V = d[l] @ b
        Tl = T[l].double().cpu().numpy()
        want_dX = want_dX + d[l][rows] @ wl + s * mask[rows] * (V[rows] @ a)
        lim_dX = lim_dX + np.abs(d[l][rows]) @ np.abs(wl) + s * mask[rows] * (np.abs(d[l][rows]) @ np.abs(b) @ np.abs(a))
        within(grads[2 * l], s * (V.T @ (x * mask)), s * ((np.abs(d[l]) @ np.abs(b)).T @ (np.abs(x) * mask)), N + 3 * M, "dA")
        within(grads[2 * l + 1], s * (d[l].T @ Tl), s * (np.abs(d[l]).T @ np.abs(Tl)), K + 3 * M, "dB")
    within(dX[t.from_numpy(rows).cuda()], want_dX, lim_dX, 4 * N + 8 * r, "dX")


@pytest.mark.parametrize("M,K", [(16, 4416), (16, 4480), (16, 4544), (11, 6528), (8, 2048), (8, 2112), (3, 5312)])
@pytest.mark.parametrize("r", [8, 136])
def test_few_tokens_about_the_room_for_them(M, K, r):
    """X that just fits, or just does not, where the kernels of few tokens keep it."""
    print(f"few tokens M={M} K={K} r={r}", flush=True)
    check_gated(Case(M, 40, K, r, 2, 0.1, seed=31))


def test_outputs_past_32_bits():
    """fp32 outputs of more than 2^31 bytes, sampled rows against the oracle."""
    import torch as t
    print("outputs past 32 bits", flush=True)
    M, wide, r, p, s = 70001, 8192, 8, 0.1, 2.0
    dev = t.Generator("cuda").manual_seed(5)
    rows = np.array([0, 1, 32767, 65535, 65536, 69887, 69888, 70000])
    at = t.from_numpy(rows).cuda()

    def bf(*shape, scale=1.0):
        return (t.randn(*shape, generator=dev, device="cuda") * scale).to(t.bfloat16)

    def f64(x):
        return x.double().cpu().numpy()

    # Y [M, 8192] from K = 64, then dX [M, 8192] of a layer with 64 rows
    for N, K in ((wide, 64), (64, wide)):
        w = G.gpu_quantize(t.randn(N, K, generator=dev, device="cuda") * 0.1)
        W, A, B, drop = f64(G.gpu_dequantize(w)), bf(r, K, scale=0.1), bf(N, r, scale=0.1), q.Dropout(p, 3, 4)
        X, size = bf(M, K), q.qlora_dropout_linear_sizes(N, K, M, r)
        mask = ref.keep(M, K, p, 3, 4)[rows]
        if N == wide:
            Y = t.empty(M, N, device="cuda")
            q.qlora_dropout_linear_fwd(w, X, A, B, r, s * r, drop, Y, None, q.workspace(size["fwd_ws_bytes"]))
            want, lim = (ref.forward(f64(X[at]), W, f64(A), f64(B), s, mask, a)[0] for a in (False, True))
            within(Y[at], want, lim, 2 * K + 4 * r, "Y")
            del Y
        else:
            dY, dX, dA, dB = bf(M, N), t.empty(M, K, device="cuda"), t.empty(r, K, device="cuda"), t.empty(N, r, device="cuda")
            q.qlora_dropout_linear_bwd(w, X, dY, A, B, r, s * r, drop, None, dX, dA, dB, q.workspace(size["bwd_ws_bytes"]))
            want, lim = (ref.backward(f64(X[at]), f64(dY[at]), W, f64(A), f64(B), s, mask, None, a)[0] for a in (False, True))
            within(dX[at], want, lim, 2 * N + 4 * r, "dX")
