"""Refusals and sizes of the layer with dropout and of the gated block on the
CPU (the pointers are fake; only validation paths run)."""

import ctypes

import pytest

import quantized_fine_tuning_amd as q

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced
BIG = 1 << 40
INVALID, DTYPE, SMALL = q.QLORA_ERR_INVALID_ARG, q.QLORA_ERR_UNSUPPORTED_DTYPE, q.QLORA_ERR_WORKSPACE_TOO_SMALL


def weight(n=256, k=256, codes=FAKE):
    return q.qlora_nf4_t(n, k, codes, FAKE, FAKE, FAKE)


def dropout(p=0.1, step=None):
    return q.qlora_dropout_t(p, 5, 6, step)


def adapters(Ag=FAKE, Bg=FAKE, Au=FAKE, Bu=FAKE, r=16, alpha=32.0):
    return q.qlora_gated_adapters_t(Ag, Bg, Au, Bu, r, alpha)


def ref(x):
    return None if x is None else ctypes.byref(x)


def linear(W=weight(), X=FAKE, m=64, A=FAKE, B=FAKE, r=16, drop=dropout(), Y=FAKE, yd=q.QLORA_BF16, T=None, ws=FAKE,
           size=BIG):
    return q.lib.qlora_dropout_linear_fwd(ref(W), X, m, A, B, r, 32.0, ref(drop), Y, yd, T, ws, size, None)


def linear_backward(W=weight(), X=FAKE, dY=FAKE, m=64, A=FAKE, B=FAKE, r=16, drop=dropout(), T=None, dX=FAKE,
                    yd=q.QLORA_BF16, dA=FAKE, dB=FAKE, ws=FAKE, size=BIG):
    return q.lib.qlora_dropout_linear_bwd(ref(W), X, dY, m, A, B, r, 32.0, ref(drop), T, dX, yd, dA, dB, ws, size, None)


def gated(W=weight(), up=weight(), X=FAKE, m=64, ad=adapters(), act=q.QLORA_ACT_SILU, drop=dropout(), H=FAKE, G=FAKE,
          U=FAKE, T=None, ws=FAKE, size=BIG):
    return q.lib.qlora_gated_fwd(ref(W), ref(up), X, m, ref(ad), act, ref(drop), H, G, U, T, ws, size, None)


def gated_backward(W=weight(), up=weight(), X=FAKE, dH=FAKE, G=FAKE, U=FAKE, m=64, ad=adapters(), act=q.QLORA_ACT_SILU,
                   drop=dropout(), T=None, dX=FAKE, yd=q.QLORA_BF16, dAg=FAKE, dBg=FAKE, dAu=FAKE, dBu=FAKE, ws=FAKE,
                   size=BIG):
    return q.lib.qlora_gated_bwd(ref(W), ref(up), X, dH, G, U, m, ref(ad), act, ref(drop), T, dX, yd, dAg, dBg, dAu, dBu,
                                 ws, size, None)


SIZES = (q.lib.qlora_dropout_linear_sizes, q.lib.qlora_gated_sizes)


@pytest.mark.parametrize("n,k,m,r,expect", [
    (256, 256, 64, 16, q.QLORA_OK),
    (8, 64, 0, 8, q.QLORA_OK),
    (256, 256, 64, 256, q.QLORA_OK),
    (256, 96, 64, 16, INVALID),
    (250, 256, 64, 16, INVALID),
    (256, 256, -1, 16, INVALID),
    (256, 256, 64, 12, INVALID),
    (256, 256, 64, 0, INVALID),
    (256, 256, 64, 264, INVALID),
    (256, 256, 1 << 24, 16, INVALID),
])
def test_sizes(n, k, m, r, expect):
    for f in SIZES:
        out = q.qlora_block_sizes_t()
        assert f(n, k, m, r, ctypes.byref(out)) == expect, q.lib.qlora_last_error()
        assert f(n, k, m, r, None) == INVALID


@pytest.mark.parametrize("n,k,r", [(4096, 4096, 16), (11008, 4096, 64), (264, 320, 24), (8, 64, 256), (2048, 5504, 8)])
def test_workspaces_cover_every_smaller_batch(n, k, r):
    """Sizes of M_max hold for each M below it: a call with exactly that many
    bytes passes the check (it then stops at the next one, a NULL workspace)."""
    W = weight(n, k)
    for m_max in (1, 16, 17, 50, 64, 65, 200, 777, 1025, 2049, 4500):
        one, two = q.qlora_dropout_linear_sizes(n, k, m_max, r), q.qlora_gated_sizes(n, k, m_max, r)
        for m in sorted({*range(1, 68), 127, 128, 129, 192, 193, 255, 256, 257, 319, 320, 321, 511, 512, 513, 600, 767, 768,
                         769, 777, 1024, 1025, 1500, 2047, 2048, 2049, 3000, 4095, 4096, 4097, 4500}):
            if m > m_max:
                break
            assert linear(W=W, m=m, r=r, ws=None, size=one["fwd_ws_bytes"]) == INVALID, (m_max, m)
            assert linear_backward(W=W, m=m, r=r, ws=None, size=one["bwd_ws_bytes"]) == INVALID, (m_max, m)
            ad = adapters(r=r)
            assert gated(W=W, up=W, m=m, ad=ad, ws=None, size=two["fwd_ws_bytes"]) == INVALID, (m_max, m)
            assert gated_backward(W=W, up=W, m=m, ad=ad, ws=None, size=two["bwd_ws_bytes"]) == INVALID, (m_max, m)


SHARED = [
    ({"W": None}, INVALID),
    ({"W": weight(250)}, INVALID),
    ({"W": weight(codes=None)}, INVALID),
    ({"X": None}, INVALID),
    ({"X": FAKE + 2}, INVALID),
    ({"m": -1}, INVALID),
    ({"m": 1 << 23}, INVALID),
    ({"T": FAKE + 4}, INVALID),
    ({"ws": None}, INVALID),
    ({"ws": FAKE + 8}, INVALID),
    ({"size": 0}, SMALL),
    ({"drop": dropout(-0.1)}, INVALID),
    ({"drop": dropout(1.0)}, INVALID),
    ({"drop": dropout(1.0 - 2.0 ** -18)}, INVALID),  # (65536 of 65536 pieces)
    ({"drop": dropout(float("nan"))}, INVALID),
    ({"drop": dropout(step=FAKE + 4)}, INVALID),
]
OF_ONE = [
    ({"A": None}, INVALID),
    ({"A": FAKE + 8}, INVALID),
    ({"B": None}, INVALID),
    ({"B": FAKE + 2}, INVALID),
    ({"r": 0}, INVALID),
    ({"r": 20}, INVALID),
    ({"r": 264}, INVALID),
    ({"yd": q.QLORA_F16}, DTYPE),
    ({"yd": 9}, DTYPE),
]
OF_TWO = [
    ({"up": None}, INVALID),
    ({"up": weight(264)}, INVALID),
    ({"up": weight(256, 320)}, INVALID),
    ({"up": weight(codes=FAKE + 4)}, INVALID),
    ({"ad": None}, INVALID),
    ({"ad": adapters(Ag=None)}, INVALID),
    ({"ad": adapters(Bg=FAKE + 8)}, INVALID),
    ({"ad": adapters(Au=FAKE + 2)}, INVALID),
    ({"ad": adapters(Bu=None)}, INVALID),
    ({"ad": adapters(r=12)}, INVALID),
    ({"act": 0}, INVALID),
    ({"act": 3}, INVALID),
    ({"G": None}, INVALID),
    ({"U": None}, INVALID),
    ({"G": FAKE + 2}, INVALID),
    ({"U": FAKE + 4}, INVALID),
]


@pytest.mark.parametrize("change,expect", SHARED + OF_ONE + [({"Y": None}, INVALID), ({"Y": FAKE + 4}, INVALID)])
def test_linear_refusals(change, expect):
    assert linear(**change) == expect, q.lib.qlora_last_error()
    assert q.lib.qlora_last_error().decode().startswith("qlora_dropout_linear_fwd: ")


@pytest.mark.parametrize("change,expect", SHARED + OF_ONE + [
    ({"dY": None}, INVALID), ({"dY": FAKE + 2}, INVALID), ({"dX": None}, INVALID), ({"dX": FAKE + 8}, INVALID),
    ({"dA": None}, INVALID), ({"dA": FAKE + 4}, INVALID), ({"dB": None}, INVALID), ({"dB": FAKE + 8}, INVALID)])
def test_linear_backward_refusals(change, expect):
    assert linear_backward(**change) == expect, q.lib.qlora_last_error()


@pytest.mark.parametrize("change,expect", SHARED + OF_TWO + [({"H": None}, INVALID), ({"H": FAKE + 8}, INVALID)])
def test_gated_refusals(change, expect):
    assert gated(**change) == expect, q.lib.qlora_last_error()
    assert q.lib.qlora_last_error().decode().startswith("qlora_gated_fwd: ")


@pytest.mark.parametrize("change,expect", SHARED + OF_TWO + [
    ({"yd": q.QLORA_F16}, DTYPE), ({"dH": None}, INVALID), ({"dH": FAKE + 2}, INVALID), ({"dX": None}, INVALID),
    ({"dX": FAKE + 4}, INVALID), ({"dAg": None}, INVALID), ({"dBg": FAKE + 8}, INVALID), ({"dAu": FAKE + 4}, INVALID),
    ({"dBu": None}, INVALID)])
def test_gated_backward_refusals(change, expect):
    assert gated_backward(**change) == expect, q.lib.qlora_last_error()


def test_no_tokens_need_no_forward():
    assert linear(m=0, X=None, Y=None, ws=None, size=0) == q.QLORA_OK
    assert gated(m=0, X=None, H=None, G=None, U=None, ws=None, size=0) == q.QLORA_OK


def test_binding_refuses_wrong_tensors_on_the_host():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    for bad in (dict(seed=-1), dict(seed=2 ** 64), dict(seed=0, offset=-1), dict(seed=0, offset=2 ** 64)):
        with pytest.raises(ValueError, match="outside"):
            q.Dropout(0.1, **bad)
    A, B = torch.zeros(8, 64, dtype=bf), torch.zeros(16, 8, dtype=bf)
    ad = q.GatedAdapters(A, B, A, B, 16.0)
    assert (ad.r, ad.n_rows, ad.n_cols) == (8, 16, 64)
    for bad in ((A, B[:, :4], A, B), (A, B, A[:, :32], B), (A, B, A, B.float()), (A.half(), B, A, B), (A, B[:8], A, B),
                (None, B, A, B), (A[0], B, A, B)):
        with pytest.raises(ValueError):
            q.GatedAdapters(*bad, 16.0)
    W, other = q.Nf4Tensor.empty(16, 64, device="cpu"), q.Nf4Tensor.empty(24, 64, device="cpu")
    X, H, ws = torch.zeros(5, 64, dtype=bf), torch.zeros(5, 16, dtype=bf), torch.zeros(1 << 12, dtype=torch.uint8)
    drop = q.Dropout(0.1, 1)
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_gated_fwd(W, W, X, ad, "silu", drop, H, None, None, None, ws)
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_dropout_linear_fwd(W, X, A, B, 8, 16.0, drop, H, None, ws)
    with pytest.raises(ValueError, match="act"):
        q.qlora_gated_fwd(W, W, X, ad, "relu", drop, H, None, None, None, ws)
    with pytest.raises(ValueError, match="up is"):
        q.qlora_gated_fwd(W, other, X, ad, "silu", drop, H, None, None, None, ws)
    for bad in (X[:, :32], X.float(), torch.zeros(64, 5, dtype=bf).t(), None, X[0]):
        with pytest.raises(ValueError):
            q.qlora_gated_fwd(W, W, bad, ad, "silu", drop, H, None, None, None, ws)
        with pytest.raises(ValueError):
            q.qlora_dropout_linear_fwd(W, bad, A, B, 8, 16.0, drop, H, None, ws)
    with pytest.raises(ValueError):
        q.qlora_dropout_linear_bwd(W, X, H, A, B, 8, 16.0, drop, None, X, torch.zeros(8, 64, dtype=bf), torch.zeros(16, 8),
                                   ws)
