"""The tiled kernels of the 8-bit products and weight gradients (fp8_layouts) on operands in wider buffers
whose padding, and what lies right behind the last row, is NaN."""
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


