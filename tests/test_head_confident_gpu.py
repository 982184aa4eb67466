"""Tokens that the model is sure of.  The log-sum-exp and the target's logit come from
one and the same sum, so nothing of the logit's rounding is left in a loss near 0:
the loss is never negative, and the target's gradient vanishes with it."""
import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from head_cases import BF16, CASES
from test_embedding_gpu import gen, rand, strided

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def sure(n, vocab, dim, dtype, logit, seed):
    """H whose logit at the label is about `logit`, the others about logit / sqrt(dim) N(0, 1)."""
    g = gen(seed)
    W = rand(g, (vocab, dim), dtype, 1.0)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    y[0], y[-1] = 0, vocab - 1
    w = W[y].float()
    H = (logit * w / (w * w).sum(1, keepdim=True)).to(dtype)
    return H, W, y, torch.full((n,), 1 / n, device="cuda")


def check(loss, want, scale=1.0):
    """No rounding of the logits (60 has a unit of 4e-6) is left: the sum of the
    exponentials is 1 and what it rounds to, 2^-23 relative and as much again for
    the logarithm."""
    assert bool((loss >= 0).all()), float(loss.min())
    assert float(want.max()) <= 1e-8
    assert float((loss.double() - want).max()) <= 2.0 ** -22 * scale, float(loss.max())


def vanish(got, n, W, H):
    """Gradients of rows whose every delta is at most `got[0]` / n in size: by the sums
    of magnitudes, far below the 2e-5 / n that a logit's rounding would leave."""
    d, dH, dW = got
    assert float(dH.abs().max()) <= d / n * float(W.abs().max()) * 2
    assert float(dW.abs().max()) <= d * float(H.abs().max()) * 2


@pytest.mark.parametrize("name", CASES)
def test_cross_entropy(gpu, name):
    dt, n, vocab, dim, _, _ = CASES[name]
    H, W, y, dloss = sure(n, vocab, dim, BF if dt == BF16 else F32, 60.0, n + dim)
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, dW = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
    torch.cuda.synchronize()
    want = R.head(H, W, labels=y)
    check(loss, want["loss"])
    R.check(lse, want["lse"], want["b_lse"], "lse")
    vanish((2.0 ** -22 + 1e-8, dH, dW), n, W, H)


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("name", CASES)
def test_distillation(gpu, name, T):
    """One stored entry: p = 1.  The backward call's q is exp(z / T - lse) with lse
    rounded to fp32, half a unit of its size, 2^-24 lse, and the quotient's rounding."""
    dt, n, vocab, dim, _, _ = CASES[name]
    H, W, y, dloss = sure(n, vocab, dim, BF if dt == BF16 else F32, 60.0 * T, n + dim)
    t = torch.full((n, 1), 3.5, device="cuda")
    loss, lse, z = mo.topk_distill_forward(H, W, y[:, None], t, temperature=T)
    dH, dW = mo.topk_distill_backward(H, W, y[:, None], t, lse, z, dloss, temperature=T)
    torch.cuda.synchronize()
    want = R.head(H, W, ids=y[:, None], teacher=t, T=T)
    check(loss, want["loss"], T * T)
    R.check(lse, want["lse"], want["b_lse"], "lse")
    vanish((T * (2.0 ** -23 * float(lse.abs().max()) + 2.0 ** -22), dH, dW), n, W, H)


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("dt", [BF, F32])
def test_strided_rows_and_masked_positions(gpu, dt, pad):
    """Operands that are copied or read as they lie; every third position masked, some
    of its H infinite."""
    H, W, y, _ = sure(150, 700, 128, dt, 60.0, 5)
    y[::3] = -1
    H[0], H[3] = float("inf"), float("nan")
    H, W = strided(H, pad, pad // 3)[0], strided(W, pad, pad // 2)[0]
    loss, lse = mo.softmax_xent_forward(H, W, y)
    ids = torch.stack([y, torch.full_like(y, -7)], 1)
    kl, l2, z = mo.topk_distill_forward(H, W, ids, torch.zeros(150, 2, device="cuda"))
    torch.cuda.synchronize()
    for x, l in ((loss, lse), (kl, l2)):
        assert bool((x[::3] == 0).all()) and bool((l[::3] == 0).all())
        assert bool((x >= 0).all()) and float(x.max()) <= 2.0 ** -22
    assert bool((z[:, 1] == 0).all()) and bool((z[::3] == 0).all())


@pytest.mark.parametrize("dt,n,vocab,dim", [(BF, 257, 32001, 2048), (BF, 37, 5000, 4096), (F32, 40, 5000, 1000), (F32, 600, 5000, 1000)])
def test_small_losses_keep_their_digits(gpu, dt, n, vocab, dim):
    """Losses of 1e-6 to 1e-2: each rival's logit is off by its sum's rounding (at most
    dim 2^-23 of the products' magnitudes; that enters as a factor), and the
    logarithm's argument by units of 2^-23."""
    H, W, y, _ = sure(n, vocab, dim, dt, 18.0, 7)
    loss, lse = mo.softmax_xent_forward(H, W, y)
    torch.cuda.synchronize()
    want = R.head(H, W, labels=y)
    assert 1e-6 < float(want["loss"].median()) < 1e-2
    err = (loss.double() - want["loss"]).abs()
    h, w = H.double(), W.double()
    dz = dim * 2.0 ** -23 * (h.abs() @ w.abs().t()).amax(1) * (6 if dt == F32 else 1)
    assert bool((err <= want["loss"] * (2 * dz + 2.0 ** -20) + 2.0 ** -22).all()), float(err.max())
