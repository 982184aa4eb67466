"""Calls the documentation allows that the operators' other tests leave out: sorts of
16385 to 32768 positions in one workgroup, with keys and positions that fill their
32-bit words; a thousand teacher entries; streams that are none; hidden states that
autograd made."""
import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand, token_sets

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("kind", ["uniform", "one", "zipf", "padded", "none"])
@pytest.mark.parametrize("n", [16384, 16385, 32767, 32768, 32769])
@pytest.mark.parametrize("vocab", [300, (1 << 17) - 1, 1 << 17])
def test_one_workgroup_sorts_up_to_its_last_position(gpu, kind, n, vocab):
    """32 words per thread; 2^17 - 1 ids and the padding take 17 bits beside the 15 of a
    position, one more id 18 and the sort of several launches."""
    g = gen(n + vocab)
    tokens = token_sets(kind, n, vocab, g)
    tokens[0], tokens[-1] = vocab - 1, vocab - 1
    dY = rand(g, (n, 8), BF)
    exact, exact_bound = (x.cuda() for x in R.embed_grad(tokens.cpu(), dY.cpu(), vocab, 0.5))
    for accumulate in (False, True):
        old = rand(g, (vocab, 8), F32)
        G = old.clone()
        mo.embedding_backward(tokens, dY, G, scale=0.5, accumulate=accumulate)
        torch.cuda.synchronize()
        want, bound = exact, exact_bound
        if accumulate:
            want = want + old.double()
            bound = bound + R.U * want.abs()
        R.check(G, want, bound + R.U * want.abs(), f"G {kind}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,dim,k", [(300, 5000, 128, 1024), (700, 900, 96, 1000), (5, 40, 64, 1024)])
def test_a_thousand_entries_with_duplicates(gpu, dtype, n, vocab, dim, k):
    """More entries than the vocabulary has rows in two of the cases: every id several
    times, some absent."""
    g = gen(n + k)
    W, H = rand(g, (vocab, dim), dtype, dim ** -0.5), rand(g, (n, dim), dtype, 2.0)
    dloss = torch.randn(n, generator=g, device="cuda") / n
    ids = torch.randint(-vocab // 8, vocab + vocab // 8, (n, k), generator=g, device="cuda")
    ids[:, 1::3] = ids[:, :1]
    ids[1] = -1
    t = torch.randn((n, k), generator=g, device="cuda") * 2
    loss, lse, z = mo.topk_distill_forward(H, W, ids, t, temperature=1.25)
    dH, dW = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss, temperature=1.25)
    torch.cuda.synchronize()
    want = R.head(H, W, dloss, ids=ids, teacher=t, T=1.25)
    for x, name in ((loss, "loss"), (lse, "lse"), (dH, "dH"), (dW, "dW")):
        R.check(x, want[name], want["b_" + name], name)


@pytest.mark.parametrize("stream", ["side", object(), [1]])
def test_a_stream_of_another_kind_is_refused(gpu, stream):
    W = torch.ones(9, 16, device="cuda", dtype=BF)
    t = torch.tensor([1, 2], device="cuda")
    before = torch.cuda.current_stream()
    with pytest.raises((TypeError, ValueError)):
        mo.embedding_forward(t, W, stream=stream)
    assert torch.cuda.current_stream() == before and torch.cuda.current_device() == 0
    Y = mo.embedding_forward(t, W)
    torch.cuda.synchronize()
    assert bool((Y == 1).all())


def test_gradients_meet_autograd_by_hand(gpu):
    """The calls are outside autograd: what they return has no grad_fn, also from
    tensors that require gradients.  The layers between them, in autograd, take and
    give gradients at the two ends."""
    g = gen(3)
    n, vocab, dim = 50, 200, 64
    W = torch.nn.Parameter(rand(g, (vocab, dim), F32, 0.1))
    A = torch.nn.Parameter(rand(g, (dim, dim), F32, dim ** -0.5))
    t, y = (torch.randint(0, vocab, (n,), generator=g, device="cuda") for _ in range(2))
    dloss = torch.full((n,), 1 / n, device="cuda")
    x = mo.embedding_forward(t, W, scale=8.0)
    assert x.grad_fn is None and not x.requires_grad
    x.requires_grad_()
    h = torch.tanh(x @ A)
    loss, lse = mo.softmax_xent_forward(h, W, y)
    dh, G = mo.softmax_xent_backward(h, W, y, loss, lse, dloss)
    assert loss.grad_fn is None and dh.grad_fn is None
    h.backward(dh)
    mo.embedding_backward(t, x.grad, G, scale=8.0, accumulate=True)
    torch.cuda.synchronize()
    W64, A64 = W.detach().double().requires_grad_(), A.detach().double().requires_grad_()
    z = torch.tanh(8.0 * W64[t] @ A64) @ W64.t()
    torch.nn.functional.cross_entropy(z, y).backward()
    # fp32 sums of at most `vocab` terms on the way
    for got, want in ((G, W64.grad), (A.grad, A64.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 2 * vocab * R.U


@pytest.mark.parametrize("n", [1000, 40000])
@pytest.mark.parametrize("vocab", [300, 5000, (1 << 18) - 1, 1 << 18, (1 << 20) + 3, 1 << 27])
@pytest.mark.parametrize("accumulate", [False, True])
def test_every_number_of_sorting_passes(gpu, n, vocab, accumulate):
    """9 bits of the ids a pass: one pass to four, in one workgroup where key and position
    share a word, in launches of their own otherwise; the first, the last and absent ids."""
    g = gen(n + vocab % 1000)
    tokens = token_sets("padded", n, vocab, g)
    tokens[:4] = torch.tensor([vocab - 1, 0, vocab, -1], device="cuda")
    dY = rand(g, (n, 3), BF)
    G = torch.full((vocab, 3), 0.5, device="cuda", dtype=BF)
    mo.embedding_backward(tokens, dY, G, accumulate=accumulate)
    torch.cuda.synchronize()
    ok = ((tokens >= 0) & (tokens < vocab)).cpu()
    ids, at = tokens.cpu()[ok].unique(return_inverse=True)
    want, bound = R.embed_grad(at, dY.cpu()[ok], len(ids), 1.0)
    if accumulate:
        want = want + 0.5
        bound = bound + R.U * want.abs()
    R.check(G[ids.cuda()].cpu(), want, bound + R.ut(BF) * want.abs(), "G")
    G[ids.cuda()] = 0.5 if accumulate else 0
    assert bool((G == (0.5 if accumulate else 0)).all())
