"""A batch of a million tokens: more blocks of dH and more tiles of H's transpose than
one grid holds, so the kernels walk them."""
import math

import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_a_million_tokens(gpu):
    n, vocab, dim = (1 << 20) - 5, 30, 4160
    # 64 x 16 elements of dH in a block, 64 x 64 of H in a tile; 2^20 of them in a grid
    assert n * dim // 1024 > 1 << 20 and n * dim // 4096 > 1 << 20
    g = gen(1)
    W = rand(g, (vocab, dim), BF, dim ** -0.5)
    H = torch.empty((n, dim), device="cuda", dtype=BF).normal_(generator=g)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    y[::9] = -1
    dloss = torch.full((n,), 1 / n, device="cuda")
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, dW = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
    torch.cuda.synchronize()
    # rows from all over the batch
    at = torch.cat([torch.arange(300, device="cuda"), torch.arange(n - 300, n, device="cuda"),
                    torch.randint(0, n, (2000,), generator=g, device="cuda")])
    want = R.head(H[at], W, dloss[at], labels=y[at])
    for x, k in ((loss, "loss"), (lse, "lse"), (dH, "dH")):
        R.check(x[at], want[k], want["b_" + k], k)
    exact, size = torch.zeros((vocab, dim), dtype=torch.float64, device="cuda"), 0.0
    w = W.double()
    for a in range(0, n, 1 << 16):
        h, t = H[a:a + (1 << 16)].double(), y[a:a + (1 << 16)]
        d = torch.softmax(h @ w.t(), 1)
        d[torch.arange(len(t), device="cuda"), t.clamp(min=0)] -= 1
        d = torch.where((t >= 0)[:, None], d / n, torch.zeros_like(d))
        exact += d.t() @ h
        size += float(((d * d).sum(1) * (h * h).sum(1)).sum())
    own = float((exact.to(BF).double() - exact).norm())
    # delta's rounding, a step of 2^-7 on [1, 2): at most 2^-8 / sqrt(3) of each term on
    # average, independent ones; 5 % for the fp32 sums
    err = float((dW.double() - exact).norm())
    assert err <= 1.05 * math.hypot(own, 2.0 ** -8 / math.sqrt(3) * math.sqrt(size)), (err, own, math.sqrt(size))
