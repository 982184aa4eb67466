"""Each path of the 8-bit products and weight gradients (fp8_cases) against the 64-bit formulas,
with scales of their own in every block."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
import operators_ref as R
from fp8_cases import PRODUCTS, WGRADS
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def shuffled(q, s, seed):
    """Scales 2^-5 to 2^5 of what they were, so that a wrong one shows."""
    g = gen(seed)
    F.codes(s).copy_(torch.randint(122, 133, s.shape, generator=g, device="cuda"))
    return q, s


def off(t, by, pad):
    """t's rows `by` bytes off alignment, `pad` further apart; what lies around is NaN."""
    big = torch.full((t.shape[0] * (t.shape[1] + pad) + by + 16,), 0x7F, dtype=torch.uint8, device="cuda")
    v = big[by:by + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(F.codes(t))
    return v.view(t.dtype)


@pytest.mark.parametrize("case", [c for c, _ in PRODUCTS], ids=lambda c: "x".join(map(str, c)))
def test_product(gpu, case):
    m, n, k, f32, blk, by, inc = case
    g = gen(m + n + k)
    dt = F32 if f32 else BF
    A, sa = shuffled(*mo.fp8_quantize(rand(g, (m, k), BF)), 1)
    if blk == 128:
        B, sb = shuffled(*mo.fp8_quantize_weight(rand(g, (n, k), BF), need_t=False)[:2], 2)
    else:
        B, sb = shuffled(*mo.fp8_quantize(rand(g, (n, k), BF)), 2)
    want, bound = F.matmul(A, sa, B, sb, 1, blk, dt)
    if by:
        A = off(A, by, 0)
    if inc:
        sa = F.codes(sa).t().contiguous().view(F.SCALE).t()
    big = torch.full((m + 1, n + 3), 7.0, device="cuda", dtype=dt)
    out = big[:m, :n]
    R.check(mo.fp8_matmul(A, sa, B, sb, out=out), want, bound, "Y")
    rel = float((out.double() - want).norm() / want.norm())
    assert rel <= (R.ut(dt) if dt == BF else 2e-6), rel
    again = mo.fp8_matmul(A, sa, B, sb, dtype=dt)
    assert torch.equal(again, out)
    out.fill_(7)
    assert bool((big == 7).all())


@pytest.mark.parametrize("case", [c for c, _ in WGRADS], ids=lambda c: "x".join(map(str, c)))
def test_weight_grad(gpu, case):
    t, n, k, f32, by = case
    g = gen(t + n + k)
    q, s = shuffled(*mo.fp8_quantize(rand(g, (t, k), BF)), 3)
    dY = rand(g, (t, n), F32 if f32 else BF)
    want, bound = F.wgrad(dY, q, s, F32)
    if by:
        big = torch.full((t * n + 16,), float("nan"), device="cuda", dtype=dY.dtype)
        v = big[by:by + t * n].view(t, n)
        v.copy_(dY)
        dY = v
    G = torch.full((n + 1, k + 3), 7.0, device="cuda")
    out = G[:n, :k]
    R.check(mo.fp8_weight_grad(dY, q, s, out), want, bound, "G")
    assert float((out.double() - want).norm() / want.norm()) <= 2e-6
    again = mo.fp8_weight_grad(dY, q, s, torch.empty((n, k), device="cuda"))
    assert torch.equal(again, out)
    out.fill_(7)
    assert bool((G == 7).all())
    old = rand(g, (n, k), BF)
    want, bound = F.wgrad(dY, q, s, BF, old)
    R.check(mo.fp8_weight_grad(dY, q, s, old.clone(), accumulate=True), want, bound, "G added")


def test_bad_values_of_an_fp32_gradient(gpu):
    """An infinity, a NaN and float32's largest in dY (three bf16 planes) reach the sums they are in alone."""
    t, n, k = 70, 33, 48
    q, s = mo.fp8_quantize(rand(gen(4), (t, k), BF))
    F.codes(q)[2:5] = 0x38
    dY = rand(gen(5), (t, n), F32)
    dY[2, 3], dY[3, 7], dY[4, 11] = float("inf"), float("nan"), torch.finfo(F32).max
    x = F.value(q, s)
    want = dY.double().t() @ x
    G = mo.fp8_weight_grad(dY, q, s, torch.empty((n, k), device="cuda")).double()
    assert torch.equal(torch.isnan(G), torch.isnan(want))
    assert bool((G[3] == want[3]).all())
    ok = torch.isfinite(want) & (want.abs() < torch.finfo(F32).max)
    assert bool(((G - want).abs()[ok] <= 1e-5 * (dY.double().abs().t() @ x.abs())[ok]).all())
