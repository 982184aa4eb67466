"""The operators together, as a training step uses them: an embedding, a layer norm
and an output head tied to the embedding, whose gradients go straight into the
buffers that the Muon step and the AdamW tail read; on other streams, and
captured in a graph."""
import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
N, V, D = 200, 1000, 256


class Model:
    """x = scale W[t]; h = norm(x); loss = mean cross entropy of h W^T."""

    def __init__(self, dtype, seed=1):
        g = gen(seed)
        self.W = rand(g, (V, D), dtype, 0.05)
        self.G = torch.zeros_like(self.W)
        self.M = torch.zeros(V, D, device="cuda")
        self.tail = torch.cat([torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")])
        self.tail_g = torch.zeros_like(self.tail)
        self.m, self.v = torch.zeros_like(self.tail), torch.zeros_like(self.tail)
        self.tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
        self.labels = torch.randint(0, V, (N,), generator=g, device="cuda")
        self.labels[::9] = -100
        valid = (self.labels >= 0).float()
        self.dloss = valid / valid.sum()
        self.loss = torch.zeros(N, device="cuda")

    def gradients(self, stream=None):
        s = dict(stream=stream)
        w, b = self.tail[:D], self.tail[D:]
        x = mo.embedding_forward(self.tokens, self.W, scale=4.0, **s)
        h, mean, rstd = mo.layer_norm_forward(x, w, b, **s)
        _, lse = mo.softmax_xent_forward(h, self.W, self.labels, loss=self.loss, **s)
        dh, _ = mo.softmax_xent_backward(h, self.W, self.labels, self.loss, lse, self.dloss, dW=self.G, **s)
        dx, _, _ = mo.layer_norm_backward(dh, x, mean, rstd, w, dweight=self.tail_g[:D], dbias=self.tail_g[D:], **s)
        mo.embedding_backward(self.tokens, dx, self.G, scale=4.0, accumulate=True, **s)

    def update(self, t):
        mo.muon_owner_step([(self.W, self.G, self.M)], lr=0.02, ns_dtype="f32" if self.W.dtype == F32 else "bf16")
        mo.adamw_tail_step(self.tail, self.tail_g, self.m, self.v, t, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                           weight_decay=0.01)

    def state(self):
        return [self.loss, self.G, self.tail_g, self.W, self.tail]


def test_gradients_of_the_whole_step_by_differences(gpu):
    """fp32: the tied matrix's gradient (head plus embedding) and the tail's against
    central differences of the 64-bit loss; step 1e-6 along a random direction.
    The chain's fp32 error stays below 1e-4 of the products' magnitudes (each
    operator's own is below 1e-5); the differences' truncation is far smaller."""
    m = Model(F32)
    m.gradients()
    torch.cuda.synchronize()
    eps = torch.tensor(1e-5, dtype=F32).double().item()

    def f(W, tail):
        x = R.embed(m.tokens, W, 4.0)
        h, _, _ = R.norm(x, tail[:D], tail[D:], eps)
        return float((R.head(h, W, labels=m.labels)["loss"] * m.dloss.double()).sum())

    g = gen(8)
    for grad, k in ((m.G, 0), (m.tail_g, 1)):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        p, q = [m.W.double(), m.tail.double()], [m.W.double(), m.tail.double()]
        p[k], q[k] = p[k] + 1e-6 * v, q[k] - 1e-6 * v
        num = (f(*p) - f(*q)) / 2e-6
        assert abs(float((grad.double() * v).sum()) - num) <= 1e-4 * float((grad.double() * v).abs().sum())


def test_training_steps_run(gpu):
    """Steps of the whole loop keep every value finite and move the weights."""
    m = Model(BF)
    before = m.W.clone()
    for t in range(1, 4):
        m.gradients()
        m.update(t)
    torch.cuda.synchronize()
    for x in m.state():
        assert bool(torch.isfinite(x).all())
    assert not torch.equal(before, m.W)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_side_streams_give_the_same_bits(gpu, dtype):
    ref = Model(dtype)
    ref.gradients()
    torch.cuda.synchronize()
    for as_handle in (False, True):
        got = Model(dtype)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got.gradients(side.cuda_stream if as_handle else side)
        churn = [torch.full((1 << 20,), float(k), device="cuda") for k in range(8)]
        del churn
        torch.cuda.synchronize()
        for a, b in zip(ref.state(), got.state()):
            assert torch.equal(a, b)


def test_two_models_on_two_streams_at_once(gpu):
    refs = [Model(BF, s) for s in (1, 2)]
    for m in refs:
        m.gradients()
    torch.cuda.synchronize()
    got = [Model(BF, s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in got]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for m, s in zip(got, streams):
            m.gradients(s)
    torch.cuda.synchronize()
    for a, b in zip(refs, got):
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_step_replays(gpu, dtype):
    """The gradients captured once; before each replay the inputs change in place.
    Every replay equals the eager call, with eager work and synchronisations
    between."""
    m, e = Model(dtype), Model(dtype)
    m.gradients()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.gradients()
    for r in range(4):
        g = gen(100 + r)
        for x in (m, e):
            g.manual_seed(100 + r)
            x.tokens.copy_(torch.randint(-1, V, (N,), generator=g, device="cuda"))
            x.labels.copy_(torch.randint(-1, V, (N,), generator=g, device="cuda"))
            x.W.copy_(rand(g, (V, D), dtype, 0.05))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e.gradients()
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        del junk
        for a, b in zip(m.state(), e.state()):
            assert torch.equal(a, b), f"replay {r}"


def test_captured_distillation_replays(gpu):
    g = gen(3)
    H, W, dloss = rand(g, (70, 128), BF), rand(g, (900, 128), BF, 0.1), torch.full((70,), 1 / 70, device="cuda")
    ids = torch.randint(-1, 900, (70, 12), generator=g, device="cuda")
    t = rand(g, (70, 12), F32, 2.0)

    def step():
        loss, lse, z = mo.topk_distill_forward(H, W, ids, t, temperature=2.0)
        dH, dW = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss, temperature=2.0)
        return loss, dH, dW

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(3):
        H.copy_(rand(g, (70, 128), BF))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), f"replay {r}"


def test_a_stream_of_another_kind_and_a_bad_workspace_are_refused(gpu):
    m = Model(BF)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(mo.MoError, match="WORKSPACE"):
        mo.embedding_backward(m.tokens, m.W[:N], m.G, workspace=small)
    with pytest.raises(ValueError, match="uint8"):
        mo.embedding_backward(m.tokens, m.W[:N], m.G, workspace=torch.empty(1 << 24, device="cuda"))
    with pytest.raises(mo.MoError, match="ALIAS"):
        mo.softmax_xent_backward(m.W[:N], m.W, m.labels, m.loss, m.loss, m.dloss, dW=m.W, need_dH=False)


def test_phases_are_timed(gpu):
    m = Model(BF)
    mo.profile_enable(True)
    try:
        mo.profile_read()
        m.gradients()
        got = mo.profile_read()
    finally:
        mo.profile_enable(False)
    for name in ("emb_fwd", "emb_sort", "emb_bwd", "ln_fwd", "ln_bwd", "hd_prep", "hd_target", "hd_lse", "hd_delta",
                 "hd_step", "hd_dh"):
        assert got[name][1] > 0 and got[name][0] > 0, name
