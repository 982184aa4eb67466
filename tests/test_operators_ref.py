"""The 64-bit reference forms of the operators, pinned on the CPU: against torch's
own float64 functions, and their gradients against central differences."""
import math

import pytest
import torch
import torch.nn.functional as F

import operators_ref as R


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def directional(f, x, dx, h=1e-6):
    """(f(x + h dx) - f(x - h dx)) / 2 h, truncation and cancellation about 1e-9."""
    return (f(x + h * dx) - f(x - h * dx)) / (2 * h)


def test_embedding_gradient_by_differences():
    tokens = torch.tensor([3, 0, 3, -1, 7, 9, 2])          # -1 and 9: padding
    W, dW, dY = rnd(8, 5), rnd(8, 5, seed=1), rnd(7, 5, seed=2)
    G, _ = R.embed_grad(tokens, dY, 8, 1.7)
    num = directional(lambda w: (R.embed(tokens, w, 1.7) * dY).sum(), W, dW)
    assert abs(float((G * dW).sum() - num)) < 1e-7
    assert bool((G[[1, 4, 5, 6]] == 0).all())
    want = F.embedding(tokens.clamp(0, 7), W) * 1.7
    want[[3, 5]] = 0
    assert torch.equal(R.embed(tokens, W, 1.7), want)


@pytest.mark.parametrize("affine", [True, False])
def test_norm_and_gradients(affine):
    X, dY = rnd(6, 11), rnd(6, 11, seed=1)
    w, b = (rnd(11, seed=2), rnd(11, seed=3)) if affine else (None, None)
    y, mu, r = R.norm(X, w, b, 1e-5)
    assert torch.allclose(y, F.layer_norm(X, (11,), w, b, 1e-5), rtol=1e-12, atol=1e-12)
    (dx, dw, db), _ = R.norm_grad(dY, X, mu, r, w)
    ddx = rnd(6, 11, seed=4)
    num = directional(lambda x: (R.norm(x, w, b, 1e-5)[0] * dY).sum(), X, ddx)
    assert abs(float((dx * ddx).sum() - num)) < 1e-7
    if affine:
        v = rnd(11, seed=5)
        assert abs(float((dw * v).sum() - directional(lambda t: (R.norm(X, t, b, 1e-5)[0] * dY).sum(), w, v))) < 1e-7
        assert abs(float((db * v).sum() - directional(lambda t: (R.norm(X, w, t, 1e-5)[0] * dY).sum(), b, v))) < 1e-7


def head_case(kind):
    H, W, dloss = rnd(7, 6), rnd(13, 6, seed=1), rnd(7, seed=2)
    if kind == "xent":
        return H, W, dloss, dict(labels=torch.tensor([0, 12, 5, -100, 13, 5, 2]))
    ids = torch.tensor([[0, 3, 12], [5, 5, 1], [-1, 2, 99], [-1, -1, 13], [4, 6, 8], [7, -1, 7], [1, 2, 3]])
    teacher = rnd(7, 3, seed=3) * 2
    teacher[4] = torch.tensor([1.0, -math.inf, 2.0])
    teacher[6] = -math.inf
    teacher[2, 0] = math.nan                                 # an absent entry's logit
    return H, W, dloss, dict(ids=ids, teacher=teacher, T=1.7)


@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_head_gradients_by_differences(kind):
    H, W, dloss, kw = head_case(kind)
    o = R.head(H, W, dloss, **kw)
    f = lambda h, w: (R.head(h, w, **kw)["loss"] * dloss).sum()
    dH, dW = rnd(7, 6, seed=7), rnd(13, 6, seed=8)
    assert abs(float((o["dH"] * dH).sum() - directional(lambda h: f(h, W), H, dH))) < 1e-6
    assert abs(float((o["dW"] * dW).sum() - directional(lambda w: f(H, w), W, dW))) < 1e-6
    dead = ~o["live"]
    assert dead.tolist() == ([False] * 3 + [True, True, False, False] if kind == "xent"
                             else [False] * 3 + [True, False, False, True])
    assert bool((o["loss"][dead] == 0).all()) and bool((o["dH"][dead] == 0).all())


def test_head_against_torch():
    H, W, _, kw = head_case("xent")
    lab = kw["labels"]
    want = F.cross_entropy(H @ W.t(), torch.where((lab >= 0) & (lab < 13), lab, -100), ignore_index=-100, reduction="none")
    assert torch.allclose(R.head(H, W, **kw)["loss"], want, rtol=1e-12, atol=1e-12)
    # every vocabulary entry stored: the plain divergence between two softmaxes
    t = rnd(7, 13, seed=5)
    ids = torch.arange(13).repeat(7, 1)
    got = R.head(H, W, ids=ids, teacher=t, T=2.0)["loss"]
    want = 4 * F.kl_div(F.log_softmax(H @ W.t() / 2, 1), F.log_softmax(t / 2, 1), log_target=True, reduction="none").sum(1)
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)


def split(x):
    """The three bf16 parts of fp32 values, each the nearest to what is left."""
    hi = x.to(torch.bfloat16)
    r = x - hi.float()
    mid = r.to(torch.bfloat16)
    lo = (r - mid.float()).to(torch.bfloat16)
    return hi, mid, lo


def test_fp32_values_are_three_bf16_parts():
    x = torch.randn(200000, generator=torch.Generator().manual_seed(1)) * 10.0 ** torch.linspace(-20, 20, 200000)
    x = torch.cat([x, torch.tensor([1.0, 1 + 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -8, 1 + 2.0 ** -9, 0.0])])
    hi, mid, lo = split(x)
    assert torch.equal(hi.double() + mid.double() + lo.double(), x.double())
    assert bool((mid.float().abs() <= 2.0 ** -8 * x.abs()).all())
    assert bool((lo.float().abs() <= 2.0 ** -16 * x.abs()).all())
