"""The RMS norm and the 8-bit operators together, as a training step uses them: a block of two
linear layers in 8 bits behind a norm with a residual, whose weights' gradients go
straight into the buffers that the Muon step reads; on other streams, captured in a
graph, and on matrices of more than 2^32 elements."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# tokens, width, inner width: small products, odd ones, a few tokens, K in parts, copied and transposed operands
SIZES = [(200, 256, 512), (70, 200, 330), (5, 384, 256), (1100, 256, 640), (4100, 1000, 1500)]


class Block:
    """h = x + res; n = norm(h); u = n W1^T; a = max(u, 0)^2; y = h + a W2^T; loss = sum(y * t)."""

    def __init__(self, tokens, dim, inner, seed=1, gdtype=BF):
        g = gen(seed)
        self.x, self.res, self.t = (rand(g, (tokens, dim), BF) for _ in range(3))
        self.w = 1 + 0.1 * rand(g, (dim,), F32)
        self.dw = torch.zeros(dim, device="cuda")
        self.W = [rand(g, (inner, dim), BF, dim ** -0.5), rand(g, (dim, inner), BF, inner ** -0.5)]
        self.G = [torch.full_like(w, float("nan"), dtype=gdtype) for w in self.W]
        self.M = [torch.zeros_like(w, dtype=F32) for w in self.W]

    def step(self, stream=None):
        s = dict(stream=stream)
        on = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.current_stream()
        w8 = [mo.fp8_quantize_weight(w, **s) for w in self.W]
        n, ns, self.h, r = mo.rms_norm_quantize(self.x, self.w, residual=self.res, **s)
        self.u = mo.fp8_matmul(n, ns, *w8[0][:2], **s)
        with torch.cuda.stream(on):
            pos = self.u.clamp(min=0)
            act = pos * pos
        a, as_ = mo.fp8_quantize(act, **s)
        self.out = mo.fp8_matmul(a, as_, *w8[1][:2], **s)
        # backward: the loss reaches h both past the layers and through them
        mo.fp8_weight_grad(self.t, a, as_, self.G[1], **s)
        t, ts = mo.fp8_quantize(self.t, **s)
        self.da = mo.fp8_matmul(t, ts, *w8[1][2:], **s)
        with torch.cuda.stream(on):
            self.du = 2 * pos * self.da
        mo.fp8_weight_grad(self.du, n, ns, self.G[0], **s)
        d, ds = mo.fp8_quantize(self.du, **s)
        self.dn = mo.fp8_matmul(d, ds, *w8[0][2:], **s)
        self.dx, _ = mo.rms_norm_backward(self.dn, self.h, r, self.w, dH=self.t, dweight=self.dw, **s)
        self.kept = w8, (n, ns), (a, as_), (t, ts), (d, ds), r

    def state(self):
        return [self.h, self.u, self.out, self.da, self.dn, self.dx, self.dw, *self.G]


@pytest.mark.parametrize("size", SIZES)
def test_the_whole_step(gpu, size):
    """Each value against the formula of its own inputs; then the gradients against those of the
    64-bit block without any rounding to 8 bits."""
    m = Block(*size)
    m.step()
    w8, n, a, t, d, r = m.kept
    for got, x, w in ((m.u, n, w8[0][:2]), (m.out, a, w8[1][:2]), (m.da, t, w8[1][2:]), (m.dn, d, w8[0][2:])):
        R.check(got, *F.matmul(*x, *w, 1, 128, BF), "product")
    R.check(m.G[0], *F.wgrad(m.du, *n, BF), "G1")
    R.check(m.G[1], *F.wgrad(m.t, *a, BF), "G2")
    (dx, dw), (b, bw) = F.rms_grad(m.dn, m.h, r, m.w, m.t)
    R.check(m.dx, dx, b, "dx")
    R.check(m.dw, dw, bw, "dw")
    # 8 bits: half a step is at most 2^-4 of a value, so 0.036 of it in the mean over a step.  Two operands: 0.05
    # of a product; the square doubles u's, and with a's and W2's own 0.11 for what is linear in a (G2 has the
    # square's and a's); da 0.05, du with u's 0.07, G1 with n's 0.08, dn with du's and W1's 0.09.  Doubled.
    h = (m.x.double() + m.res.double()).requires_grad_()
    W = [w.double().requires_grad_() for w in m.W]
    w = m.w.double().requires_grad_()
    nn = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w
    y = h + (nn @ W[0].t()).clamp(min=0).square() @ W[1].t()
    (y * m.t.double()).sum().backward()
    for got, want, what in ((m.G[0], W[0].grad, "G1"), (m.G[1], W[1].grad, "G2"), (m.dx, h.grad, "dx"), (m.dw, w.grad, "dw")):
        off = float((got.double() - want).norm() / want.norm())
        assert off < 0.22, (what, off)


def test_training_steps_run(gpu):
    """The owner step on the written gradients moves the weights and leaves every value finite."""
    m = Block(*SIZES[0])
    before = [w.clone() for w in m.W]
    for _ in range(3):
        m.step()
        mo.muon_owner_step(list(zip(m.W, m.G, m.M)), lr=0.02, ns_dtype="bf16")
    torch.cuda.synchronize()
    for x in m.state() + m.W:
        assert bool(torch.isfinite(x).all())
    assert not any(torch.equal(a, b) for a, b in zip(before, m.W))


@pytest.mark.parametrize("size", SIZES)
def test_calls_repeat_bit_by_bit_and_on_side_streams(gpu, size):
    ref = Block(*size)
    ref.step()
    ref.step()
    torch.cuda.synchronize()
    again = Block(*size)
    again.step()
    side = Block(*size)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side.step(s)
    churn = [torch.full((1 << 20,), float(k), device="cuda") for k in range(8)]
    del churn
    torch.cuda.synchronize()
    for a, b, c in zip(ref.state(), again.state(), side.state()):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_two_blocks_on_two_streams_at_once(gpu):
    size = SIZES[3]
    refs = [Block(*size, seed=k) for k in (1, 2)]
    for m in refs:
        m.step()
    torch.cuda.synchronize()
    got = [Block(*size, seed=k) for k in (1, 2)]
    streams = [torch.cuda.Stream() for _ in got]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for m, s in zip(got, streams):
            m.step(s)
    torch.cuda.synchronize()
    for a, b in zip(refs, got):
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("size", SIZES)
def test_captured_step_replays(gpu, size):
    """Captured once; before each replay the inputs change in place.  Every replay equals the eager
    call, with eager work and synchronisations between."""
    m, e = Block(*size), Block(*size)
    m.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    for r in range(4):
        for b in (m, e):
            g = gen(100 + r)
            for t in (b.x, b.res, b.t, *b.W):
                t.copy_(rand(g, t.shape, BF, 0.3 + r))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e.step()
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        del junk
        for a, b in zip(m.state(), e.state()):
            assert torch.equal(a, b), f"replay {r}"


def test_two_graphs_share_a_workspace(gpu):
    """Two captured products on one caller's workspace, replayed in turn on one stream."""
    g = gen(5)
    A = [mo.fp8_quantize(rand(g, (1500, 16384), BF)) for _ in range(2)]
    B = [mo.fp8_quantize_weight(rand(g, (1000, 16384), BF), need_t=False)[:2] for _ in range(2)]
    need = mo.fp8_matmul_workspace_bytes(*A[0], *B[0])
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = [torch.empty((1500, 1000), device="cuda", dtype=BF) for _ in range(2)]
    want = [mo.fp8_matmul(*a, *b) for a, b in zip(A, B)]
    torch.cuda.synchronize()
    graphs = []
    for a, b, o in zip(A, B, out):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            mo.fp8_matmul(*a, *b, out=o, workspace=ws)
    for _ in range(4):
        ws.fill_(255)
        for o in out:
            o.zero_()
        for x in graphs:
            x.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("tokens", [1, 2, 3, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65])
@pytest.mark.parametrize("n,k", [(17, 1), (40, 127), (129, 2176), (1000, 640), (4096, 130)])
def test_few_tokens(gpu, tokens, n, k):
    g = gen(1000 * tokens + n + k)
    A = mo.fp8_quantize(rand(g, (tokens, k), F32))
    B = mo.fp8_quantize_weight(rand(g, (n, k), F32), need_t=False)[:2]
    for dt in (BF, F32):
        R.check(mo.fp8_matmul(*A, *B, dtype=dt), *F.matmul(*A, *B, 1, 128, dt), str(dt))


def test_a_matrix_with_itself(gpu):
    """Reads may be of one and the same matrix; a written one is refused."""
    A, s = mo.fp8_quantize(rand(gen(6), (300, 512), BF))
    R.check(mo.fp8_matmul(A, s, A, s), *F.matmul(A, s, A, s, 1, 1, BF), "A A^T")
    x = rand(gen(7), (64, 128), BF)
    w = torch.ones(128, device="cuda")
    assert torch.equal(mo.rms_norm_forward(x, w, residual=x)[1], x + x)
    y, _, r = mo.rms_norm_forward(x, w)
    assert torch.equal(mo.rms_norm_backward(x, x, r, w, dH=x)[0], mo.rms_norm_backward(x, x.clone(), r, w, dH=x.clone())[0])
    for call in (lambda: mo.rms_norm_forward(x, w, out=x), lambda: mo.rms_norm_forward(x, w, residual=y, h=x),
                 lambda: mo.rms_norm_backward(y, x, r, w, dX=y),
                 lambda: mo.fp8_dequantize(A, s, out=A.view(torch.uint8).view(BF))):
        with pytest.raises((mo.MoError, ValueError)):
            call()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(mo.MoError, match="WORKSPACE"):
        mo.rms_norm_backward(y, x, r, w, workspace=small)


def test_phases_are_timed(gpu):
    m = Block(*SIZES[4])
    mo.profile_enable(True)
    try:
        mo.profile_read()
        m.step()
        got = mo.profile_read()
    finally:
        mo.profile_enable(False)
    for name in ("rn_fwd", "rn_bwd", "f8_cast", "f8_prep", "f8_gemm", "f8_wgrad"):
        assert got[name][1] > 0 and got[name][0] > 0, name


def test_rows_beyond_2_32_elements(gpu):
    """Norm, casts and a product of (2^20 - 3) x 4224: the last rows as alone."""
    rows, cols, last = (1 << 20) - 3, 4224, 500
    g = gen(9)
    x = torch.empty((rows, cols), device="cuda", dtype=BF)
    x.normal_(generator=g)
    w = 1 + 0.1 * rand(g, (cols,), F32)
    tail = x[-last:].contiguous()
    q, s, _, r = mo.rms_norm_quantize(x, w)
    qt, st, _, rt = mo.rms_norm_quantize(tail, w)
    assert torch.equal(F.codes(q[-last:]), F.codes(qt)) and torch.equal(F.codes(s[-last:]), F.codes(st))
    assert torch.equal(r[-last:], rt)
    dX, dw = mo.rms_norm_backward(x, x, r, w, need_dweight=False)
    assert torch.equal(dX[-last:], mo.rms_norm_backward(tail, tail, rt, w, need_dweight=False)[0])
    del dX
    q, s = mo.fp8_quantize(x)
    back = mo.fp8_dequantize(q, s)
    qt, st = mo.fp8_quantize(tail)
    assert torch.equal(F.codes(q[-last:]), F.codes(qt))
    assert torch.equal(back[-last:], mo.fp8_dequantize(qt, st))
    del back, x
    B = mo.fp8_quantize_weight(rand(g, (70, cols), BF), need_t=False)[:2]
    for dt in (BF, F32):
        Y = mo.fp8_matmul(q, s, *B, dtype=dt)
        R.check(Y[-last:], *F.matmul(qt, st, *B, 1, 128, dt), str(dt))
        Y = mo.fp8_matmul(B[0], B[1], q, s, dtype=dt)
        R.check(Y[:, -last:], *F.matmul(*B, qt, st, 128, 1, dt), str(dt))
    # a weight gradient to which only the last tokens give anything
    for dt in (BF, F32):
        dY = torch.zeros((rows, 40), device="cuda", dtype=dt)
        dY[-last:] = rand(g, (last, 40), dt)
        G = torch.empty((40, cols), device="cuda")
        R.check(mo.fp8_weight_grad(dY, q, s, G), *F.wgrad(dY[-last:], qt, st, F32), "G")


def test_a_result_beyond_2_32_elements(gpu):
    m, n, k, last = 70001, 65664, 128, 300
    g = gen(10)
    A, sa = mo.fp8_quantize(rand(g, (m, k), BF))
    B, sb, _, _ = mo.fp8_quantize_weight(rand(g, (n, k), BF), need_t=False)
    Y = mo.fp8_matmul(A, sa, B, sb)
    R.check(Y[-last:], *F.matmul(A[-last:], sa[-last:], B, sb, 1, 128, BF), "Y")
    del Y
    dY, n2 = rand(g, (64, m), BF), 65664
    q, s = mo.fp8_quantize(rand(g, (64, n2), BF))
    G = torch.empty((m, n2), device="cuda", dtype=BF)
    mo.fp8_weight_grad(dY, q, s, G)
    want, bound = F.wgrad(dY[:, -last:], q, s, BF)
    R.check(G[-last:], want, bound, "G")


@pytest.mark.parametrize("m,n,k", [(5, 300, 512), (70, 300, 640), (70, 300, 600), (300, 256, 1024)])
def test_scales_at_both_ends(gpu, m, n, k):
    """The least scales (down to bf16's subnormal numbers) against the largest: products as of any
    others.  Where values are taken as bf16 numbers, one below 2^-130 is rounded to a multiple of 2^-133
    (bf16's last step; a value has four bits), so it is off by 2^-134 at most."""
    A, sa = mo.fp8_quantize(rand(gen(11), (m, k), F32))
    B, sb = mo.fp8_quantize(rand(gen(12), (n, k), F32))
    a = F.codes(A)
    a[(a & 0x7F) < 8] = 0
    g = gen(13)
    F.codes(sa).copy_(torch.randint(0, 3, sa.shape, generator=g, device="cuda"))
    F.codes(sb).copy_(torch.randint(225, 240, sb.shape, generator=g, device="cuda"))
    off = 2.0 ** -134 * F.value(B, sb).abs().sum(1)
    for dt in (BF, F32):
        Y, bound = F.matmul(A, sa, B, sb, 1, 1, dt)
        bound = bound + off * (1 + R.ut(dt))
        R.check(mo.fp8_matmul(A, sa, B, sb, dtype=dt), Y, bound, str(dt))
        R.check(mo.fp8_matmul(B, sb, A, sa, dtype=dt), Y.t(), bound.t(), str(dt))
    dY = rand(gen(14), (m, 200), BF) * 2.0 ** 110
    off = 2.0 ** -134 * dY.double().abs().sum(0)[:, None]
    for y in (dY, dY.float()):
        G, bound = F.wgrad(y, A, sa, F32)
        R.check(mo.fp8_weight_grad(y, A, sa, torch.empty((200, k), device="cuda")), G, bound + off, "G")
