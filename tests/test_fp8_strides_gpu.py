"""8-bit products and weight gradients at the longest strides that the entry points accept: offsets inside
a tile up to 2^31, addresses beyond 2^32.  What lies between the rows is never written to or summed."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def apart(t, ld):
    """t with rows ld elements apart (the gaps as the allocator left them)."""
    rows, cols = t.shape
    v = torch.empty((rows - 1) * ld + cols, dtype=t.dtype, device=t.device).as_strided((rows, cols), (ld, 1))
    v.copy_(t)
    return v


def far(q, s, ld, lds):
    return apart(F.codes(q), ld).view(F.FP8), apart(F.codes(s), lds).view(F.SCALE)


def eight(seed, rows, cols, blk=1):
    x = rand(gen(seed), (rows, cols), BF)
    return mo.fp8_quantize(x) if blk == 1 else mo.fp8_quantize_weight(x, need_t=False)[:2]


@pytest.mark.parametrize("m,n,k,dtype,blk,ld,lds", [
    (1030, 2600, 2048, BF, 128, (1 << 23) - 16, (1 << 23) - 4),   # tiles in 8 bits, in place
    (1030, 2600, 2048, BF, 1, (1 << 23) - 16, (1 << 23) - 4),
    (1030, 2600, 640, F32, 128, (1 << 23) - 1, (1 << 23) - 1),    # as values
    (70, 300, 500, BF, 1, (1 << 23) - 1, (1 << 23) - 1)])         # small
def test_product(gpu, m, n, k, dtype, blk, ld, lds):
    A, B = eight(1, m, k), eight(2, n, k, blk)
    want, bound = F.matmul(*A, *B, 1, blk, dtype)
    R.check(mo.fp8_matmul(*far(*A, ld, lds), *far(*B, ld, lds), dtype=dtype), want, bound, "Y")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("t,n,k,dtype,ldy,ld,lds", [
    (300, 1504, 2048, BF, (1 << 24) - 8, (1 << 25) - 16, (1 << 25) - 1),   # in place, tiles of 64, 128 and 256
    (70, 2600, 2048, BF, (1 << 24) - 8, (1 << 25) - 16, (1 << 25) - 1),
    (70, 2600, 4112, BF, (1 << 24) - 8, (1 << 25) - 16, (1 << 25) - 1),
    (70, 9000, 1101, BF, (1 << 26) - 1, 1 << 26, 1 << 26),                 # transposed first
    (70, 1504, 8016, F32, (1 << 26) - 1, 1 << 26, 1 << 26),
    (65, 129, 257, BF, 1 << 26, 1 << 26, 1 << 26), (65, 129, 257, F32, 1 << 26, 1 << 26, 1 << 26)])   # small
def test_weight_grad(gpu, t, n, k, dtype, ldy, ld, lds):
    q, s = eight(3, t, k)
    dY = rand(gen(4), (t, n), dtype)
    want, bound = F.wgrad(dY, q, s, F32)
    G = mo.fp8_weight_grad(apart(dY, ldy), *far(q, s, ld, lds), torch.empty((n, k), device="cuda"))
    R.check(G, want, bound, "G")
    torch.cuda.empty_cache()
