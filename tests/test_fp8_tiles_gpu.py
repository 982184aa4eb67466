"""The tiled kernels of the 8-bit products and weight gradients (fp8_layouts) at what they are most
likely to get wrong: NaN, infinities and NaN scales, the least and the largest scales, and operands in
wider buffers whose padding, and what lies right behind the last row, is NaN."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
import operators_ref as R
from fp8_layouts import PRODUCTS, WGRADS, name
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def place(t, off, pad, fill, tail):
    """t in rows `pad` further apart from element `off` on, `tail` elements of the buffer behind the last row."""
    rows, cols = t.shape
    ld = cols + pad
    big = torch.full((off + (rows - 1) * ld + cols + tail,), fill, dtype=t.dtype, device=t.device)
    v = big.as_strided((rows, cols), (ld, 1), off)
    v.copy_(t)
    return v


def laid(q, s, lay):
    """A matrix in 8 bits in this layout, NaN (and NaN scales) around it."""
    tail = 64 * (q.shape[1] + lay.pad)   # whatever a stage of rows behind the last one would take
    v = place(F.codes(q), lay.off, lay.pad, 0x7F, tail).view(F.FP8)
    c = F.codes(s)
    if lay.cols and c.shape[1] > 1:
        w = place(c.t(), lay.soff, lay.spad, 255, 4096).t()
    else:
        w = place(c, lay.soff, lay.spad, 255, 4096)
    return v, w.view(F.SCALE)


def operand(seed, rows, cols, blk):
    x = rand(gen(seed), (rows, cols), BF)
    q, s = mo.fp8_quantize(x) if blk == 1 else mo.fp8_quantize_weight(x, need_t=False)[:2]
    F.codes(s).copy_(torch.randint(122, 133, s.shape, generator=gen(seed + 1), device="cuda"))
    return q, s


def inside(c, rows, cols, dtype):
    """A result in the middle of sevens, and a check that they are still there."""
    big = torch.full((rows + 2, cols + 5), 7.0, device="cuda", dtype=dtype)
    out = big[1:rows + 1, 2:cols + 2]

    def untouched():
        keep = out.clone()
        out.fill_(7)
        ok = bool((big == 7).all())
        out.copy_(keep)
        return ok
    return out, untouched


def product(c, A, sa, B, sb):
    dt = F32 if c.f32 else BF
    out, untouched = inside(c, c.m, c.n, dt)
    Y = mo.fp8_matmul(*laid(A, sa, c.a), *laid(B, sb, c.b), out=out)
    assert untouched()
    assert torch.equal(mo.fp8_matmul(*laid(A, sa, c.a), *laid(B, sb, c.b), dtype=dt).view(torch.int16 if dt == BF else torch.int32),
                       Y.contiguous().view(torch.int16 if dt == BF else torch.int32))
    return Y


@pytest.mark.parametrize("c", PRODUCTS, ids=name)
def test_product(gpu, c):
    dt = F32 if c.f32 else BF
    A, sa = operand(1, c.m, c.k, 1)
    B, sb = operand(3, c.n, c.k, c.blk)
    want, bound = F.matmul(A, sa, B, sb, 1, c.blk, dt)
    Y = product(c, A, sa, B, sb)
    R.check(Y, want, bound, "Y")
    off = float((Y.double() - want).norm() / want.norm())
    assert off <= (R.ut(dt) if dt == BF else 2e-6), off


@pytest.mark.parametrize("c", PRODUCTS, ids=name)
def test_product_bad_values(gpu, c):
    """NaN in an element or a scale reaches its rows and columns alone; the others stay what they are."""
    A, sa = operand(1, c.m, c.k, 1)
    B, sb = operand(3, c.n, c.k, c.blk)
    kb, r = sa.shape[1], c.blk
    rows_a, rows_b = [0, c.m // 2, c.m - 1], [3, c.n - 1]
    clean = []
    for q, bad in ((A, rows_a + [5]), (B, rows_b + list(range(r * 1, min(2 * r, c.n)) if r > 1 else [40]))):
        z = q.clone()
        F.codes(z)[bad] = 0
        clean.append((z, bad))
    F.codes(A)[rows_a[0], c.k - 1] = 0x7F
    F.codes(A)[rows_a[1], 0] = 0xFF
    F.codes(A)[rows_a[2], c.k // 2] = 0x7F
    F.codes(B)[rows_b[0], c.k - 1] = 0xFF
    F.codes(B)[rows_b[1], 70] = 0x7F
    F.codes(sa)[5, kb - 1] = 255
    F.codes(sb)[1 if r > 1 else 40, 0] = 255
    nan = torch.zeros((c.m, c.n), dtype=torch.bool, device="cuda")
    nan[clean[0][1]] = True
    nan[:, clean[1][1]] = True
    Y = product(c, A, sa, B, sb)
    assert torch.equal(torch.isnan(Y), nan)
    F.codes(sa)[5, kb - 1] = 127
    F.codes(sb)[1 if r > 1 else 40, 0] = 127
    dt = F32 if c.f32 else BF
    want, bound = F.matmul(clean[0][0], sa, clean[1][0], sb, 1, r, dt)
    R.check(torch.where(nan, want, Y.double()), want, bound, "the others")


@pytest.mark.parametrize("c", PRODUCTS, ids=name)
def test_product_scales(gpu, c):
    """Scales 2^-20 to 2^20 meet the right blocks; then the least of A's against large ones of B, and the
    other way round.  Where values are taken as bf16 numbers, one below 2^-130 is rounded to a multiple of
    2^-133 (bf16's last step; a value has four bits), so it is off by 2^-134 at most."""
    dt = F32 if c.f32 else BF
    A, sa = operand(1, c.m, c.k, 1)
    B, sb = operand(3, c.n, c.k, c.blk)
    g = gen(5)
    draw = lambda s, lo, hi: F.codes(s).copy_(torch.randint(lo, hi, s.shape, generator=g, device="cuda"))
    draw(sa, 107, 148), draw(sb, 107, 148)
    R.check(product(c, A, sa, B, sb), *F.matmul(A, sa, B, sb, 1, c.blk, dt), "far apart")
    for least, x, other, most, r in ((sa, A, B, sb, c.blk), (sb, B, A, sa, 1)):
        a = F.codes(x)
        a[(a & 0x7F) < 8] = 0
        draw(least, 0, 3), draw(most, 225, 240)
        Y, bound = F.matmul(A, sa, B, sb, 1, c.blk, dt)
        off = 2.0 ** -134 * F.value(other, most, r).abs().sum(1)
        bound = bound + (off if x is A else off[:, None]) * (1 + R.ut(dt))
        R.check(product(c, A, sa, B, sb), Y, bound, "both ends")


@pytest.mark.parametrize("m,n,k", [(64, 64, 128), (64, 200, 1024), (1030, 2600, 2048), (9000, 777, 2048)])
def test_product_of_large_terms_that_cancel(gpu, m, n, k):
    """Two products in each block that are 2^17 times the others and cancel: each of a block's products is kept to
    about 2^-17 of its largest for a bf16 result (fp8_ref's bound takes 2^-16), and exactly for an fp32 one."""
    A, B = (rand(gen(s), (r, k), F32) for s, r in ((21, m), (22, n)))
    for b in range(0, k, 128):
        A[:, b + 5], A[:, b + 100], B[:, b + 5], B[:, b + 100] = 448, -448, 448, 448
    A, B = A.to(F.FP8), B.to(F.FP8)
    sa, sb = (torch.full((r, k // 128), 127, dtype=torch.uint8, device="cuda").view(F.SCALE) for r in (m, n))
    for dt in (BF, F32):
        want, bound = F.matmul(A, sa, B, sb, 1, 1, dt)
        R.check(mo.fp8_matmul(A, sa, B, sb, dtype=dt), want, bound, str(dt))


# ---- weight gradients -------------------------------------------------------------------

def gradient(c, dY, q, s, dtype=F32, old=None):
    out, untouched = inside(c, c.n, c.k, dtype)
    if old is not None:
        out.copy_(old)
    y = place(dY, c.y[0], c.y[1], float("nan"), 64 * (c.n + c.y[1]))
    mo.fp8_weight_grad(y, *laid(q, s, c.x), out, accumulate=old is not None)
    G = out.clone()
    assert untouched()
    return G


def gradient_inputs(c):
    q, s = operand(7, c.t, c.k, 1)
    return rand(gen(9), (c.t, c.n), F32 if c.f32 else BF), q, s


@pytest.mark.parametrize("c", WGRADS, ids=name)
def test_weight_grad(gpu, c):
    dY, q, s = gradient_inputs(c)
    want, bound = F.wgrad(dY, q, s, F32)
    G = gradient(c, dY, q, s)
    R.check(G, want, bound, "G")
    assert float((G.double() - want).norm() / want.norm()) <= 2e-6
    assert torch.equal(gradient(c, dY, q, s), G)
    old = rand(gen(10), (c.n, c.k), BF)
    R.check(gradient(c, dY, q, s, BF, old), *F.wgrad(dY, q, s, BF, old), "G added")


@pytest.mark.parametrize("c", WGRADS, ids=name)
def test_weight_grad_bad_values(gpu, c):
    """Infinities, NaN, float32's largest and NaN scales reach the sums they are in and no others, from the
    first token and from the last."""
    dY, q, s = gradient_inputs(c)
    dY0, q0, t = dY.clone(), q.clone(), c.t
    dY[t - 1, 3], dY[5, 7], dY[t - 1, c.n - 1] = float("inf"), float("nan"), -float("inf")
    if c.f32:
        dY[0, 11] = torch.finfo(F32).max
    F.codes(q)[t - 1, 9] = 0x7F
    F.codes(q)[0, c.k - 1] = 0xFF
    F.codes(s)[2, 1] = 255
    x = F.value(q, s)
    want = dY.double().t() @ x
    rows = [3, 7, c.n - 1] + ([11] if c.f32 else [])
    cols = [9, c.k - 1] + list(range(128, 256))
    G = gradient(c, dY, q, s)
    assert torch.equal(torch.isnan(G), torch.isnan(want))
    inf = torch.isinf(want) & (torch.arange(c.n, device="cuda") != 11)[:, None]
    assert torch.equal(torch.isinf(G) & (torch.arange(c.n, device="cuda") != 11)[:, None], inf)
    assert torch.equal(G.double()[inf], want[inf])
    F.codes(s)[2, 1] = 127
    good = torch.ones((c.n, c.k), dtype=torch.bool, device="cuda")
    good[rows] = False
    good[:, cols] = False
    want, bound = F.wgrad(dY0, q0, s, F32)
    R.check(torch.where(good, G.double(), want), want, bound, "the others")
    if c.f32:   # what its three parts make up, where that does not overflow
        dY0[0, 11] = torch.finfo(F32).max
        want, bound = F.wgrad(dY0, q0, s, F32)
        good[11] = want[11].abs() < torch.finfo(F32).max / 2
        good[11, cols] = False
        R.check(torch.where(good, G.double(), want)[11:12], want[11:12], bound[11:12], "float32's largest")


@pytest.mark.parametrize("c", WGRADS, ids=name)
def test_weight_grad_scales(gpu, c):
    """Tokens' scales far apart, and those of 0 (2^-127); then the least alone, against a large dY."""
    dY, q, s = gradient_inputs(c)
    g = gen(11)
    F.codes(s).copy_(torch.randint(107, 148, s.shape, generator=g, device="cuda"))
    F.codes(s)[::7] = 0
    R.check(gradient(c, dY, q, s), *F.wgrad(dY, q, s, F32), "far apart")
    F.codes(s).copy_(torch.randint(0, 3, s.shape, generator=g, device="cuda"))
    a = F.codes(q)
    a[(a & 0x7F) < 8] = 0
    dY = dY * 2.0 ** 110
    want, bound = F.wgrad(dY, q, s, F32)
    off = 2.0 ** -134 * dY.double().abs().sum(0)[:, None]
    R.check(gradient(c, dY, q, s), want, bound + off, "the least")
