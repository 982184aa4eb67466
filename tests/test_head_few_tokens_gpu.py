"""bf16 gradients of few tokens: rows of dW are a term or two, so delta's rounding would
show in them as it is.  dW is as near the 64-bit form as its own rounding to bf16."""
import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPES = [(1, 700, 128), (2, 3000, 96), (3, 300, 1024), (8, 5000, 512), (40, 300, 192), (64, 2000, 64), (65, 29746, 256),
          (100, 513, 130), (128, 30011, 233), (128, 1000, 2048)]


def weights(g, n, vocab, dim):
    """Hidden states whose label stands out, and weights of the rows that differ."""
    W = rand(g, (vocab, dim), BF, dim ** -0.5)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    H = (torch.randn((n, dim), generator=g, device="cuda") + 2 * W[y].float()).to(BF)
    return H, W, y, torch.randn(n, generator=g, device="cuda")


def near(got, want, what):
    """At most 2 % above the error of rounding `want` itself: delta in two planes is exact to
    2^-16, its sums to 2^-20."""
    own = float((want.to(BF).double() - want).norm())
    err = float((got.double() - want).norm())
    assert err <= 1.02 * own, (what, err / own)


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("n,vocab,dim", SHAPES)
def test_cross_entropy(gpu, n, vocab, dim, seed):
    H, W, y, dloss = weights(gen(seed * 1000 + n), n, vocab, dim)
    loss, lse = mo.softmax_xent_forward(H, W, y)
    _, dW = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
    torch.cuda.synchronize()
    near(dW, R.head(H, W, dloss, labels=y)["dW"], "dW")


@pytest.mark.parametrize("k", [1, 9])
@pytest.mark.parametrize("n,vocab,dim", SHAPES)
def test_distillation(gpu, n, vocab, dim, k):
    g = gen(n + k)
    H, W, y, dloss = weights(g, n, vocab, dim)
    ids = torch.randint(0, vocab, (n, k), generator=g, device="cuda")
    ids[:, 0] = y
    t = torch.randn((n, k), generator=g, device="cuda")
    loss, lse, z = mo.topk_distill_forward(H, W, ids, t, temperature=1.5)
    _, dW = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss, temperature=1.5)
    torch.cuda.synchronize()
    near(dW, R.head(H, W, dloss, ids=ids, teacher=t, T=1.5)["dW"], "dW")


def test_infinite_and_huge_weights(gpu):
    """A weight near the largest fp32 value overflows nothing on the way to dW; an
    infinite one shows in its row of dH and its label's of dW, and in no other row of dH."""
    H, W, y, dloss = weights(gen(5), 6, 300, 64)
    dloss[2] = 3e38
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, dW = mo.softmax_xent_backward(H * 2 ** -20, W, y, loss, lse, dloss)
    assert bool(torch.isfinite(dW).all())
    dloss[2] = float("inf")
    dH, dW = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
    torch.cuda.synchronize()
    keep = torch.arange(6, device="cuda") != 2
    assert bool(torch.isfinite(dH[keep]).all()) and not bool(torch.isfinite(dH[2]).any())
    assert not bool(torch.isfinite(dW[y[2]]).any())
