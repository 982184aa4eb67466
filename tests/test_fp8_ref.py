"""The 64-bit forms of the RMS norm and the 8-bit operators, pinned on the CPU: against torch's
own casts and float64 functions, and their gradients against differences and autograd."""
import pytest
import torch
import torch.nn.functional as T

import fp8_ref as F
import operators_ref as R
from test_operators_ref import directional, rnd


def test_e4m3_is_torchs_cast():
    """Every number, every middle of two, their neighbours in float32, and random values, up to 448."""
    grid = torch.arange(0, 127, dtype=torch.uint8).view(F.FP8).float()
    mid = (grid[1:] + grid[:-1]) / 2
    x = torch.cat([grid, mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1),
                   torch.randn(5000, generator=torch.Generator().manual_seed(1)) * 60])
    x = torch.cat([x, -x]).clamp(-448, 448)
    assert torch.equal(F.e4m3(x.double()), x.to(F.FP8).double())
    assert bool(torch.isnan(F.e4m3(torch.tensor([float("inf"), float("nan")]).double())).all())


def test_scales_are_the_least():
    a = torch.cat([torch.exp(torch.linspace(-90, 88, 3001, dtype=torch.float64)),
                   torch.tensor([0.0, 448.0, 448.0001, 1.75, 2.0 ** -149, 2.0 ** -119 * 1.75, 3e38], dtype=torch.float64)])
    b = F.bytes_of(a)
    assert bool(((b >= 0) & (b <= 247)).all())
    assert bool((a <= 448 * torch.exp2(b - 127)).all())
    assert bool(((a > 448 * torch.exp2(b - 128)) | (b == 0)).all())


def test_quantized_values_are_near():
    """Half a step, 2^-4 of the value, or half of the least step of the block's scale."""
    x = rnd(70, 300, seed=2) * torch.exp(rnd(70, 1, seed=3))
    for r in (1, 128):
        q, b = F.quantize(x, r)
        s = F.spread(torch.exp2(b - 127), 70, 300, r)
        assert bool(((q * s - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s)).all())
        assert bool((q.abs() <= 448).all()) and bool((F.row_amax(q)[:, :2].amax() > 224))


@pytest.mark.parametrize("affine", [True, False])
def test_rms_norm_and_gradients(affine):
    X, dY, dH = rnd(6, 11), rnd(6, 11, seed=1), rnd(6, 11, seed=7)
    w = rnd(11, seed=2) if affine else None
    y, r = F.rms(X, w, 1e-6)
    assert torch.allclose(y, T.rms_norm(X, (11,), w, 1e-6), rtol=1e-12, atol=1e-12)
    (dx, dw), _ = F.rms_grad(dY, X, r, w, dH)
    d = rnd(6, 11, seed=4)
    num = directional(lambda x: (F.rms(x, w, 1e-6)[0] * dY).sum() + (x * dH).sum(), X, d)
    assert abs(float((dx * d).sum() - num)) < 1e-7
    if affine:
        v = rnd(11, seed=5)
        assert abs(float((dw * v).sum() - directional(lambda t: (F.rms(X, t, 1e-6)[0] * dY).sum(), w, v))) < 1e-7


def test_products():
    """Against loops over the blocks' numbers and scales."""
    q, b = F.quantize(rnd(5, 200, seed=1))
    p, c = F.quantize(rnd(130, 200, seed=2), 128)
    v = lambda t: torch.exp2(t - 127)
    Y, bound = F.matmul(q, v(b), p, v(c), 1, 128, torch.float32)
    for i, j in ((0, 0), (4, 127), (3, 128), (2, 129)):
        want = sum(float(q[i, k]) * 2.0 ** (float(b[i, k // 128]) - 127) * float(p[j, k]) *
                   2.0 ** (float(c[j // 128, k // 128]) - 127) for k in range(200))
        assert abs(float(Y[i, j]) - want) < 1e-12 * 200
    dY = rnd(5, 7, seed=3).float()
    G, _ = F.wgrad(dY, q, v(b), torch.float32)
    W = rnd(7, 200, seed=4).requires_grad_()
    ((F.value(q, v(b)) @ W.t()) * dY.double()).sum().backward()
    assert torch.allclose(G, W.grad, rtol=1e-12, atol=1e-12)
