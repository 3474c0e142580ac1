"""One fine-tuning step of several adapters on one quantized head, as a program
runs it: plan, adapters_fwd to the logits, the distillation loss with its
gradient in the logits' place, adapters_bwd, AdamW on the pool; then the same
pool serves single tokens.  Every stage is checked against the fp64 oracle on
what the stage before it produced, and the whole step is captured into a graph
and replayed on new batches."""

import numpy as np
import pytest

import quantized_fine_tuning_amd as q
from oracle import adamw as ref_adamw
from oracle import adapters as ref
from tests import gpu_util as G
from tests.test_gpu_adapters import Case, within
from tests.test_gpu_distill import bounds, check

pytestmark = pytest.mark.gpu

VOCAB, N, K, R, COUNT, TOP, TAU = 501, 504, 320, 16, 3, 12, 2.0


class Step:
    def __init__(self, M):
        import torch as t
        self.c = c = Case(M, N, K, R, COUNT, "mixed", seed=11)
        g = t.Generator().manual_seed(4)
        self.index = t.from_numpy(c.index).cuda()
        self.top = t.randn(M, TOP, generator=g).cuda()
        self.at = t.stack([t.randperm(VOCAB, generator=g)[:TOP] for _ in range(M)]).to(t.int32).cuda()
        self.weight = (t.rand(M, generator=g) / M).cuda()
        self.weight[::7] = 0.0
        e = lambda *s, dtype=t.float32: t.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        self.Z, self.T = e(M, N, dtype=t.bfloat16), e(M, R)
        self.loss, self.dX = e(M), e(M, K, dtype=t.bfloat16)
        self.dA, self.dB = e(COUNT, R, K), e(COUNT, N, R)
        self.moments = [t.zeros_like(x) for x in (self.dA, self.dA, self.dB, self.dB)]
        self.wsf, self.wsb = c.scratch("fwd_ws_bytes"), c.scratch("bwd_ws_bytes")

    def forward(self):
        c = self.c
        q.qlora_adapters_plan(self.index, c.plan)
        q.qlora_adapters_fwd(c.w, c.X, c.pool, c.plan, self.Z, self.T, self.wsf)

    def gradient(self):
        q.qlora_distill_fwd(self.Z, self.top, self.at, TAU, self.weight, self.loss, None, self.Z, vocab=VOCAB)

    def backward(self):
        c = self.c
        q.qlora_adapters_bwd(c.w, c.X, self.Z, c.pool, c.plan, self.T, self.dX, self.dA, self.dB, self.wsb)

    def update(self, step):
        c, m = self.c, self.moments
        q.qlora_adamw_step([(c.A, self.dA, m[0], m[1]), (c.B, self.dB, m[2], m[3])], 1e-2, 0.9, 0.999, 1e-8, 0.01, step)

    def run(self, step=1):
        self.forward()
        self.gradient()
        self.backward()
        self.update(step)


@pytest.mark.parametrize("M", [9, 40, 150, 300])
def test_each_stage_on_what_the_one_before_gave(M):
    import torch as t
    s = Step(M)
    c = s.c
    X, _, A, B, scale = c.host
    s.forward()
    want, _ = ref.forward(X, c.W, A, B, scale, c.index)
    size, _ = ref.forward(X, c.W, A, B, scale, c.index, absolute=True)
    within(s.Z, want, size, 2 * K + 4 * R, "logits", 2.0 ** -8)
    logits = s.Z.clone()
    s.gradient()
    (loss, _, dZ), lim = bounds(logits.cpu(), s.top.cpu(), s.at.cpu(), TAU, s.weight.cpu(), VOCAB)
    check(s.loss, loss, lim[0], "f32", "loss")
    check(s.Z, dZ, lim[2], "bf16", "dZ")
    assert not s.Z[:, VOCAB:].any()
    s.backward()
    dY, T = s.Z.double().cpu().numpy(), s.T.double().cpu().numpy()
    want = ref.backward(X, dY, c.W, A, B, scale, c.index, T)
    size = ref.backward(X, dY, c.W, A, B, scale, c.index, T, absolute=True)
    within(s.dX, want[0], size[0], 2 * N + 4 * R, "dX", 2.0 ** -8)
    within(s.dA, want[1], size[1], N + 3 * M, "dA")
    within(s.dB, want[2], size[2], K + 3 * M, "dB")
    for name, p, grad in (("A", c.A, s.dA), ("B", c.B, s.dB)):
        setattr(s, "before_" + name, (G.host_bf16(p).copy(), grad.cpu().numpy()))
    s.update(1)
    for name, p in (("A", c.A), ("B", c.B)):
        bits, grad = getattr(s, "before_" + name)
        zeros = np.zeros(grad.size, np.float32)
        want, _, _ = ref_adamw.step(bits.reshape(-1), grad.reshape(-1), zeros, zeros, 1e-2, 0.9, 0.999, 1e-8, 0.01, 1,
                                    param_bf16=True)
        np.testing.assert_array_equal(G.host_bf16(p).reshape(-1), want)
    # the updated pool serves single tokens
    few = q.AdapterPlan.empty(3, COUNT)
    index = np.array([2, -1, 0], np.int32)
    q.qlora_adapters_plan(t.from_numpy(index).cuda(), few)
    Y = t.full((3, N), float("nan"), device="cuda")
    q.qlora_adapters_fwd(c.w, c.X[:3], c.pool, few, Y, None, s.wsf)
    A, B = c.A.double().cpu().numpy(), c.B.double().cpu().numpy()
    want, _ = ref.forward(X[:3], c.W, A, B, scale, index)
    size, _ = ref.forward(X[:3], c.W, A, B, scale, index, absolute=True)
    within(Y, want, size, 2 * K + 4 * R, "served tokens")


@pytest.mark.parametrize("M", [40, 200])
def test_the_step_in_a_graph(M):
    """Replays, each on another batch, against the eager step from the same state."""
    import torch as t
    s = Step(M)
    state = [s.c.A, s.c.B, *s.moments]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        s.run()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        s.run()
    g = t.Generator(device="cuda").manual_seed(8)
    for rep in range(3):
        print(f"adapter step M={M} replay {rep}", flush=True)
        s.index.copy_(t.randint(-1, COUNT, (M,), generator=g, device="cuda", dtype=t.int32))
        s.c.X.copy_(t.randn(M, K, generator=g, device="cuda"))
        kept = [x.clone() for x in state]
        s.run()
        t.cuda.synchronize()
        want = [x.clone() for x in (*state, s.loss, s.dX)]
        for x, k in zip(state, kept):
            x.copy_(k)
        for x in (s.Z, s.T, s.loss, s.dX, s.dA, s.dB):
            x.fill_(float("nan"))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip((*state, s.loss, s.dX), want))
