"""Refusals of the log-probability entry points on the CPU (the pointers are
fake; only validation paths run)."""

import pytest

import quantized_fine_tuning_amd as q

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced
INVALID, DTYPE = q.QLORA_ERR_INVALID_ARG, q.QLORA_ERR_UNSUPPORTED_DTYPE

SHARED = [
    ({"zd": 7}, DTYPE),
    ({"zd": -1}, DTYPE),
    ({"m": -1}, INVALID),
    ({"m": 1 << 22}, INVALID),
    ({"v": 0}, INVALID),
    ({"v": 1001}, INVALID),
    ({"ld": 1 << 28}, INVALID),
    ({"tau": 0.0}, INVALID),
    ({"tau": float("nan")}, INVALID),
    ({"tau": 1e7}, INVALID),
    ({"Z": None}, INVALID),
    ({"Z": FAKE + 2}, INVALID),
    ({"target": None}, INVALID),
    ({"target": FAKE + 4}, INVALID),
    ({"g": FAKE + 4}, INVALID),
    ({"h": FAKE + 8}, INVALID),
    ({"dZ": FAKE + 8}, INVALID),
    ({"g": None, "h": None}, INVALID),
]


def forward(Z=FAKE, zd=q.QLORA_BF16, m=4, v=1000, ld=1000, target=FAKE, tau=1.0, logp=FAKE, lse=FAKE, ent=FAKE, k=4,
            tl=FAKE, ti=FAKE, g=FAKE, h=FAKE, dZ=FAKE):
    return q.lib.qlora_logprobs_fwd(Z, zd, m, v, ld, target, tau, logp, lse, ent, k, tl, ti, g, h, dZ, None)


def backward(Z=FAKE, zd=q.QLORA_BF16, m=4, v=1000, ld=1000, target=FAKE, tau=1.0, lse=FAKE, ent=FAKE, g=FAKE, h=FAKE,
             dZ=FAKE):
    return q.lib.qlora_logprobs_bwd(Z, zd, m, v, ld, target, tau, lse, ent, g, h, dZ, None)


@pytest.mark.parametrize("change,expect", SHARED + [
    ({"logp": None}, INVALID),
    ({"logp": FAKE + 4}, INVALID),
    ({"lse": FAKE + 4}, INVALID),
    ({"ent": FAKE + 4}, INVALID),
    ({"k": -1}, INVALID),
    ({"k": q.QLORA_LOGPROBS_MAX_TOP + 1}, INVALID),
    ({"tl": None}, INVALID),
    ({"ti": None}, INVALID),
    ({"ti": FAKE + 4}, INVALID),
])
def test_forward_refusals(change, expect):
    assert forward(**change) == expect, change


@pytest.mark.parametrize("change,expect", SHARED + [
    ({"lse": None}, INVALID),
    ({"ent": None}, INVALID),
    ({"dZ": None}, INVALID),
])
def test_backward_refusals(change, expect):
    assert backward(**change) == expect, change


def test_no_tokens():
    """M = 0 needs no pointers and launches nothing."""
    assert forward(m=0, Z=None, target=None, logp=None, lse=None, ent=None, tl=None, ti=None, g=None, h=None,
                   dZ=None) == q.QLORA_OK
    assert backward(m=0, Z=None, target=None, lse=None, ent=None, g=None, h=None, dZ=None) == q.QLORA_OK


def test_binding_refuses_wrong_tensors_on_the_host():
    torch = pytest.importorskip("torch")
    Z, t, f = torch.zeros(4, 24), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    top, at = torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int32)
    for bad in ((Z.double(), t), (Z[0], t), (Z, t.long()), (Z, t[:3]), (Z.t(), t)):
        with pytest.raises(ValueError):
            q.qlora_logprobs_fwd(bad[0], bad[1], 1.0, f)
        with pytest.raises(ValueError):
            q.qlora_logprobs_bwd(bad[0], bad[1], 1.0, f, f, Z)
    for bad in ({"lse": f[:3]}, {"entropy": f.double()}, {"top_logp": top}, {"top_index": at},
                {"top_logp": top, "top_index": at.long()}, {"top_logp": top, "top_index": at[:, :2]}, {"d_logp": f[:2]},
                {"d_entropy": f.half()}, {"dZ": Z.half(), "d_logp": f}, {"dZ": Z[:, :8], "d_logp": f}):
        with pytest.raises(ValueError):
            q.qlora_logprobs_fwd(Z, t, 1.0, f, **bad)
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_logprobs_fwd(Z, t, 1.0, f)
    with pytest.raises(ValueError):
        q.qlora_logprobs_bwd(Z, t, 1.0, f, f, None)
