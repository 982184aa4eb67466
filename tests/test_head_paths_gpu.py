"""The cross entropy and the distillation at sizes chosen for the path they take
(head_cases.py): every tile width, with several stages of K, K split or not, the
vocabulary in one piece or several, against the 64-bit forms."""
import math

import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from head_cases import BF16, CASES
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(name):
    dt, n, vocab, dim, _, _ = CASES[name]
    dt = BF if dt == BF16 else F32
    g = gen(n + vocab + dim)
    W, H = rand(g, (vocab, dim), dt, 1 / math.sqrt(dim)), rand(g, (n, dim), dt, 2.0)
    dloss = torch.randn(n, generator=g, device="cuda") / n
    dloss[1] = 0
    return g, H, W, dloss


def own_rounding(x):
    return float((x.to(BF).double() - x).norm())


def dw_bound(want, H, W, dloss, T, planes, **kw):
    """How far a bf16 dW may be from the exact one, in norm.  With delta in two planes: the
    result's own rounding (2 % for the rest).  With one plane delta is rounded too,
    divided by the significand of the largest of the first rows' T |dloss|.  The size
    of that error depends on where delta's significands lie (a step of 2^-7 on [1, 2):
    sqrt(1/12) 2^-7 of a value near 1, half of that near 2) and, of a few hundred rows,
    on chance, so it is computed from the 64-bit delta; the two errors are independent
    of each other, and 5 % allow for what is left of that and for deltas that fall on
    the other side of a tie."""
    own = own_rounding(want["dW"])
    if planes == 2:
        return 1.02 * own
    live, at, p, _ = R.targets(W.shape[0], T=T, **kw)
    h = torch.where(live[:, None], H.double(), torch.zeros_like(H, dtype=torch.float64))
    z = h @ W.double().t() / T
    c = torch.where(live, dloss.double() * T, torch.zeros_like(dloss, dtype=torch.float64))[:, None]
    delta = torch.softmax(z, 1)
    delta.scatter_add_(1, at, -p)
    delta = c * delta
    top = float((T * dloss[:64].abs()).max())
    r = 2.0 * math.frexp(top)[0]
    err = ((delta / r).to(BF).double() * r - delta).t() @ h
    return 1.05 * math.hypot(own, float(err.norm()))


def compare(got, want, H, W, dloss, name, T=1.0, **kw):
    for x, k in zip(got, ("loss", "lse", "dH", "dW")):
        R.check(x, want[k], want["b_" + k], k)
    # and the whole.  bf16: dH is made up for delta's rounding at the targets; away from them
    # delta is small, and what is left is at most the result's own rounding
    err = {k: float((x.double() - want[k]).norm()) for x, k in ((got[2], "dH"), (got[3], "dW"))}
    if H.dtype == BF:
        most = {"dH": 1.45 * own_rounding(want["dH"]),
                "dW": dw_bound(want, H, W, dloss, T, CASES[name][5].get("dt_planes", 2 if H.shape[0] <= 128 else 1), **kw)}
    else:
        # one rounding (2 u) of the sum for every 32 of K and plane pair, independent ones,
        # and lse's and the logits' own
        n, (vocab, dim) = H.shape[0], W.shape
        top = float(want["lse"].abs().max())
        most = {k: R.U * (8 + 4 * math.sqrt(6 * depth / 32) + 16 * math.sqrt(6 * dim / 32) + 8 * top) * float(want[k].norm())
                for k, depth in (("dH", vocab), ("dW", n))}
    for k in err:
        assert err[k] <= most[k], (k, err[k] / most[k])


@pytest.mark.parametrize("name", CASES)
def test_cross_entropy(gpu, name):
    g, H, W, dloss = inputs(name)
    n, vocab = H.shape[0], W.shape[0]
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    y[::7] = -100
    y[2], y[3], y[-1] = vocab - 1, 0, vocab // 2
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, dW = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
    torch.cuda.synchronize()
    compare((loss, lse, dH, dW), R.head(H, W, dloss, labels=y), H, W, dloss, name, labels=y)


@pytest.mark.parametrize("name", CASES)
def test_distillation(gpu, name):
    """Twelve entries over the whole vocabulary (every piece), one of them twice, one
    row without any."""
    g, H, W, dloss = inputs(name)
    n, vocab, k, T = H.shape[0], W.shape[0], 12, 1.5
    ids = torch.randint(0, vocab, (n, k), generator=g, device="cuda")
    ids[:, 3], ids[:, 7] = ids[:, 2], vocab - 1
    ids[::5, 6] = -1
    ids[4] = -1
    t = 2 * torch.randn((n, k), generator=g, device="cuda")
    loss, lse, z = mo.topk_distill_forward(H, W, ids, t, temperature=T)
    dH, dW = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss, temperature=T)
    torch.cuda.synchronize()
    compare((loss, lse, dH, dW), R.head(H, W, dloss, ids=ids, teacher=t, T=T), H, W, dloss, name, T, ids=ids, teacher=t)
    h, w = H.double(), W.double()
    ok = ids >= 0
    want = (h[:, None, :] * w[ids.clamp(min=0)]).sum(2) if n * k * H.shape[1] < 1 << 28 else None
    if want is not None:
        az = (h.abs()[:, None, :] * w.abs()[ids.clamp(min=0)]).sum(2)
        six = 6 if H.dtype == F32 else 1
        bound = (2 * six * H.shape[1] * R.U + (2.0 ** -22 if six == 6 else 0)) * az + R.U * want.abs()
        R.check(z[ok], want[ok], bound[ok], "z")
    assert bool((z[~ok] == 0).all())
    again = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss, temperature=T)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)
