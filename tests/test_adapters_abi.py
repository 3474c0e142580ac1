"""Refusals and sizes of the many-adapter and distillation entry points on the
CPU (the pointers are fake; only validation paths run)."""

import ctypes

import pytest

import quantized_fine_tuning_amd as q

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced
BIG = 1 << 40
INVALID, DTYPE, SMALL = q.QLORA_ERR_INVALID_ARG, q.QLORA_ERR_UNSUPPORTED_DTYPE, q.QLORA_ERR_WORKSPACE_TOO_SMALL


def weight(n=256, k=256):
    return q.qlora_nf4_t(n, k, FAKE, FAKE, FAKE, FAKE)


def pool(A=FAKE, B=FAKE, scale=FAKE, count=4, r=16):
    return q.qlora_adapters_t(A, B, scale, count, r)


@pytest.mark.parametrize("n,k,m,r,count,expect", [
    (256, 256, 64, 16, 4, q.QLORA_OK),
    (8, 64, 0, 8, 1, q.QLORA_OK),
    (256, 256, 64, 256, 1024, q.QLORA_OK),
    (256, 96, 64, 16, 4, INVALID),
    (250, 256, 64, 16, 4, INVALID),
    (256, 256, -1, 16, 4, INVALID),
    (256, 256, 64, 12, 4, INVALID),
    (256, 256, 64, 0, 4, INVALID),
    (256, 256, 64, 264, 4, INVALID),
    (256, 256, 64, 16, 0, INVALID),
    (256, 256, 64, 16, 1025, INVALID),
    (256, 256, 1 << 24, 16, 4, INVALID),
])
def test_sizes(n, k, m, r, count, expect):
    out = q.qlora_adapters_sizes_t()
    assert q.lib.qlora_adapters_sizes(n, k, m, r, count, ctypes.byref(out)) == expect, q.lib.qlora_last_error()
    if expect == q.QLORA_OK:
        assert out.plan_bytes >= 4 * (3 * m + count)
    assert q.lib.qlora_adapters_sizes(n, k, m, r, count, None) == INVALID


@pytest.mark.parametrize("n,k,r,count", [(4096, 4096, 16, 8), (11008, 4096, 64, 40), (264, 320, 24, 1000)])
def test_workspaces_cover_every_smaller_batch(n, k, r, count):
    """Sizes of M_max hold for each M below it: a call with exactly that many
    bytes passes the check (it then stops at the next one, a NULL workspace)."""
    d, ad = weight(n, k), pool(count=count, r=r)
    for m_max in (1, 16, 17, 50, 64, 200, 777, 1025, 2049):
        sizes = q.qlora_adapters_sizes(n, k, m_max, r, count)
        for m in sorted({*range(1, 66), 63, 64, 65, 129, 255, 256, 257, 511, 600, 777, 1024, 1025, 2048, 2049}):
            if m > m_max:
                break
            assert q.lib.qlora_adapters_fwd(ctypes.byref(d), FAKE, m, ctypes.byref(ad), FAKE, BIG, FAKE, q.QLORA_BF16,
                                            None, None, sizes["fwd_ws_bytes"], None) == INVALID, (m_max, m)
            assert q.lib.qlora_adapters_bwd(ctypes.byref(d), FAKE, FAKE, m, ctypes.byref(ad), FAKE, BIG, None, FAKE,
                                            q.QLORA_BF16, FAKE, FAKE, None, sizes["bwd_ws_bytes"],
                                            None) == INVALID, (m_max, m)


def test_plan_refusals():
    def call(index=FAKE, m=64, count=4, plan=FAKE, size=BIG):
        return q.lib.qlora_adapters_plan(index, m, count, plan, size, None)

    assert call(index=None) == INVALID
    assert call(index=FAKE + 4) == INVALID
    assert call(m=-1) == INVALID
    assert call(m=1 << 24) == INVALID
    assert call(count=0) == INVALID
    assert call(count=2000) == INVALID
    assert call(plan=None) == INVALID
    need = q.qlora_adapters_sizes(8, 64, 64, 8, 4)["plan_bytes"]
    assert call(size=need - 1) == SMALL


def test_forward_refusals():
    d = weight()
    args = dict(W=d, X=FAKE, m=64, ad=pool(), plan=FAKE, pb=BIG, Y=FAKE, yd=q.QLORA_BF16, T=None, ws=FAKE, wsb=BIG)

    def call(**kw):
        a = {**args, **kw}
        ref = [None if a[x] is None else ctypes.byref(a[x]) for x in ("W", "ad")]
        return q.lib.qlora_adapters_fwd(ref[0], a["X"], a["m"], ref[1], a["plan"], a["pb"], a["Y"], a["yd"], a["T"],
                                        a["ws"], a["wsb"], None)

    for kw in (dict(W=None), dict(ad=None), dict(X=None), dict(X=FAKE + 2), dict(m=-1), dict(plan=None), dict(Y=None),
               dict(T=FAKE + 4), dict(ws=None), dict(ad=pool(A=None)), dict(ad=pool(B=FAKE + 8)),
               dict(ad=pool(scale=None)), dict(ad=pool(r=20)), dict(ad=pool(count=0)), dict(m=1 << 23)):
        assert call(**kw) == INVALID, kw
    assert call(yd=q.QLORA_F16) == DTYPE
    assert call(wsb=0) == SMALL
    assert call(pb=64) == SMALL
    assert "plan" in q.lib.qlora_last_error().decode()


def test_backward_refusals():
    d, ad = weight(), pool()

    def call(X=FAKE, dY=FAKE, m=64, T=None, dX=FAKE, dxd=q.QLORA_BF16, dA=FAKE, dB=FAKE, ws=FAKE, wsb=BIG, pb=BIG):
        return q.lib.qlora_adapters_bwd(ctypes.byref(d), X, dY, m, ctypes.byref(ad), FAKE, pb, T, dX, dxd, dA, dB, ws,
                                        wsb, None)

    for kw in (dict(X=None), dict(dY=None), dict(dY=FAKE + 2), dict(dX=None), dict(dA=None), dict(dB=FAKE + 4),
               dict(T=FAKE + 8), dict(ws=None), dict(m=-2)):
        assert call(**kw) == INVALID, kw
    assert call(dxd=q.QLORA_F16) == DTYPE
    assert call(wsb=0) == SMALL
    assert call(pb=0) == SMALL


def test_distillation_refusals():
    def fwd(Z=FAKE, zd=q.QLORA_BF16, m=8, v=100, ld=104, top=FAKE, td=q.QLORA_F32, at=FAKE, k=4, tau=1.0, w=None,
            loss=FAKE, lse=None, dZ=None):
        return q.lib.qlora_distill_fwd(Z, zd, m, v, ld, top, td, at, k, tau, w, loss, lse, dZ, None)

    def bwd(lse=FAKE, dZ=FAKE, **kw):
        a = dict(Z=FAKE, zd=q.QLORA_BF16, m=8, v=100, ld=104, top=FAKE, td=q.QLORA_F32, at=FAKE, k=4, tau=1.0)
        a.update(kw)
        return q.lib.qlora_distill_bwd(*a.values(), lse, None, dZ, None)

    for f in (fwd, bwd):
        for kw in (dict(Z=None), dict(Z=FAKE + 2), dict(m=-1), dict(v=0), dict(v=105), dict(ld=1 << 31, v=5),
                   dict(top=None), dict(at=None), dict(at=FAKE + 4), dict(k=0), dict(k=513), dict(tau=0.0),
                   dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(dZ=FAKE + 2),
                   dict(m=1 << 30, ld=1 << 20)):
            assert f(**kw) == INVALID, (f, kw)
        assert f(zd=5) == DTYPE
        assert f(td=-1) == DTYPE
    assert fwd(loss=None) == INVALID
    assert fwd(w=FAKE + 4) == INVALID
    assert fwd(lse=FAKE + 8) == INVALID
    assert bwd(lse=None) == INVALID
    assert bwd(dZ=None) == INVALID
    # no tokens: nothing is enqueued and no pointer needed
    assert fwd(m=0, Z=None, top=None, at=None, loss=None) == q.QLORA_OK
    assert bwd(m=0, Z=None, top=None, at=None, lse=None, dZ=None) == q.QLORA_OK


def test_distillation_refuses_more_tokens_than_one_launch_holds():
    for m in (1 << 22, (1 << 31) - 1, 1 << 31):
        assert q.lib.qlora_distill_fwd(FAKE, q.QLORA_BF16, m, 1, 1, FAKE, q.QLORA_F32, FAKE, 1, 1.0, None, FAKE, None,
                                       None, None) == INVALID
        assert q.lib.qlora_distill_bwd(FAKE, q.QLORA_BF16, m, 1, 1, FAKE, q.QLORA_F32, FAKE, 1, 1.0, FAKE, None, FAKE,
                                       None) == INVALID


def test_binding_refuses_wrong_tensors_on_the_host():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    A, B, s = torch.zeros(3, 8, 64, dtype=bf), torch.zeros(3, 16, 8, dtype=bf), torch.zeros(3)
    p = q.AdapterPool(A, B, s)
    assert (p.count, p.r, p.n_rows, p.n_cols) == (3, 8, 16, 64)
    for bad in ((A[:2], B, s), (A, B[:, :, :4], s), (A.float(), B, s), (A, B, s.double()), (A, B, s[:2]), (A[0], B, s)):
        with pytest.raises(ValueError):
            q.AdapterPool(*bad)
    W = q.Nf4Tensor.empty(16, 64, device="cpu")
    plan = q.AdapterPlan.empty(5, 3, device="cpu")
    X, Y, ws = torch.zeros(5, 64, dtype=bf), torch.zeros(5, 16, dtype=bf), torch.zeros(1 << 12, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_adapters_fwd(W, X, p, plan, Y, None, ws)
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_adapters_fwd(W, torch.zeros(64, 5, dtype=bf).t(), p, plan, Y, None, ws)
    with pytest.raises(ValueError, match="plan"):
        q.qlora_adapters_fwd(W, X[:4], p, plan, Y[:4], None, ws)
    with pytest.raises(ValueError, match="plan"):
        q.qlora_adapters_fwd(W, X, p, q.AdapterPlan.empty(5, 4, device="cpu"), Y, None, ws)
    with pytest.raises(ValueError, match="weight"):
        q.qlora_adapters_fwd(q.Nf4Tensor.empty(24, 64, device="cpu"), X, p, plan, Y, None, ws)
    with pytest.raises(ValueError):
        q.qlora_adapters_fwd(W, X.half(), p, plan, Y, None, ws)
    with pytest.raises(ValueError):
        q.qlora_adapters_fwd(W, X, p, plan, Y.half(), None, ws)
    with pytest.raises(ValueError):
        q.qlora_adapters_plan(torch.zeros(5, dtype=torch.int64), plan)
    Z, t, at, loss = torch.zeros(4, 24), torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4)
    for bad in ((Z.double(), t, at), (Z, t[:, :2], at), (Z, t, at.long()), (Z[:3], t, at)):
        with pytest.raises(ValueError):
            q.qlora_distill_fwd(*bad, 1.0, None, loss)
    with pytest.raises(ValueError):
        q.qlora_distill_fwd(Z, t, at, 1.0, loss[:2], loss)
    with pytest.raises(ValueError):
        q.qlora_distill_fwd(Z, t, at, 1.0, None, loss, dZ=Z.bfloat16())
    with pytest.raises(ValueError):
        q.qlora_distill_bwd(Z, t, at, 1.0, None, None, Z)
