"""Forms of the C entry points that the binding does not use: an RMS norm into both results at once, without
the sum or rstd, and a weight's transposed copy alone.  Each output equals, bit by bit, that of the call
that makes it by itself, and nothing else is written."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
from matrix_optimizers_amd.operators import _code, _ptr
from test_embedding_gpu import gen, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def around(rows, cols, dtype, byte):
    """A result in the middle of bytes, and the buffer."""
    size = torch.empty(0, dtype=dtype).element_size()
    big = torch.full(((rows + 2) * (cols + 3) * size,), byte, dtype=torch.uint8, device="cuda").view(dtype).view(rows + 2, cols + 3)
    return big[1:rows + 1, 1:cols + 1], big


def untouched(out, big, byte):
    bits(out).fill_(0)
    left = bits(big).clone()
    bits(out).fill_(-1)
    other = bits(big)
    same = left == other
    inside = torch.zeros_like(same)
    inside[1:out.shape[0] + 1, 1:out.shape[1] + 1] = True
    word = int.from_bytes(bytes([byte]) * big.element_size(), "little", signed=big.element_size() > 1)
    return bool((same == ~inside).all()) and bool((left[~inside] == word).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(7, 100), (19, 256), (5, 411), (9, 512), (11, 1000), (6, 4096), (3, 4100), (4, 8192), (3, 16384),
                                       (3, 16385), (2, 20000)])
def test_rms_norm_forms(gpu, rows, cols, dtype):
    lib, stream = mo.load_library(), torch.cuda.current_stream().cuda_stream
    g, kb, es, code = gen(rows + cols), F.blocks(cols), 0x11, _code(torch.empty(0, dtype=dtype), "X")
    x, d, w = rand(g, (rows, cols), dtype), rand(g, (rows, cols), dtype), 1 + 0.1 * rand(g, (cols,), F32)
    for res in (None, d):
        y, h, r = mo.rms_norm_forward(x, w, residual=res)
        q, s, h8, r8 = mo.rms_norm_quantize(x, w, residual=res)
        assert torch.equal(r, r8) and torch.equal(h, h8)
        for with_y in (True, False):
            for with_q in (True, False):
                for with_h in ((True, False) if res is not None else (False,)):
                    for with_r in (True, False):
                        if not with_y and not with_q:
                            continue
                        made = {k: around(*sz, es) for k, sz in dict(y=(rows, cols, dtype), q=(rows, cols, F.FP8), s=(rows, kb, F.SCALE),
                                                                     h=(rows, cols, dtype)).items()}
                        rstd = torch.full((rows,), -7.0, device="cuda")
                        at = lambda k, on: (_ptr(made[k][0]), made[k][0].stride(0)) if on else (None, 0)
                        st = lib.rms_norm_forward(_ptr(x), cols, _ptr(res), cols if res is not None else 0, _ptr(w), *at("h", with_h),
                                                  *at("y", with_y), *at("q", with_q), *at("s", with_q), _ptr(rstd) if with_r else None,
                                                  rows, cols, code, 1e-6, stream)
                        assert st == 0
                        for k, on, want in (("y", with_y, y), ("q", with_q, q), ("s", with_q, s), ("h", with_h, h)):
                            out, big = made[k]
                            if on:
                                assert torch.equal(bits(out), bits(want)), (k, with_y, with_q, with_h, with_r)
                                assert untouched(out, big, es), k
                            else:
                                assert bool((big.view(torch.uint8) == es).all()), k
                        assert torch.equal(rstd, r) if with_r else bool((rstd == -7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 256), (37, 300), (300, 129), (257, 2049)])
def test_a_weights_transpose_alone(gpu, rows, cols, dtype):
    lib, stream = mo.load_library(), torch.cuda.current_stream().cuda_stream
    W = rand(gen(rows * cols), (rows, cols), dtype)
    _, _, qt, st = mo.fp8_quantize_weight(W)
    (a, abig), (b, bbig) = around(cols, rows, F.FP8, 0x11), around(F.blocks(cols), F.blocks(rows), F.SCALE, 0x11)
    assert lib.fp8_quantize_weight(_ptr(W), cols, _code(W, "W"), rows, cols, None, 0, None, 0, _ptr(a), a.stride(0), _ptr(b),
                                   b.stride(0), stream) == 0
    assert torch.equal(bits(a), bits(qt)) and torch.equal(bits(b), bits(st))
    assert untouched(a, abig, 0x11) and untouched(b, bbig, 0x11)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(7, 100), (300, 1000), (40, 8192), (9, 16400)])
def test_rms_norm_backward_forms(gpu, rows, cols, dtype):
    """dH without dX takes no part; each output alone equals itself beside the other."""
    g = gen(rows - cols)
    x, dy, dh, w = rand(g, (rows, cols), dtype), rand(g, (rows, cols), dtype), rand(g, (rows, cols), dtype), 1 + 0.1 * rand(g, (cols,), F32)
    _, _, r = mo.rms_norm_forward(x, w)
    dx, dw = mo.rms_norm_backward(dy, x, r, w, dH=dh)
    assert torch.equal(mo.rms_norm_backward(dy, x, r, w, dH=dh, need_dweight=False)[0], dx)
    for other in (None, dh):
        none, dw2 = mo.rms_norm_backward(dy, x, r, w, dH=other, need_dX=False)
        assert none is None and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [100, 1000, 8192, 16400])
def test_rms_norm_rows_out_of_range(gpu, dtype, cols):
    """Squares are fp32: a row whose sum of squares overflows has r and y 0; with eps 0 a row of zeros, or of values
    whose squares underflow, has an infinite r.  The rows beside them are as alone."""
    x = rand(gen(cols), (5, cols), dtype)
    good = x.clone()
    x[1, 3], x[2], x[3] = 1e30, 0, 1e-30
    for eps in (1e-6, 0.0):
        y, _, r = mo.rms_norm_forward(x, eps=eps)
        q, s, _, r8 = mo.rms_norm_quantize(x, eps=eps)
        assert torch.equal(r, r8)
        want = mo.rms_norm_forward(good, eps=eps)
        for i in (0, 4):
            assert torch.equal(y[i], want[0][i]) and torch.equal(r[i], want[2][i])
        assert float(r[1]) == 0 and bool((y[1] == 0).all()) and bool((q[1].float() == 0).all())
        if eps:   # (1000 to a few roundings of 2^-24: 3e-4)
            assert bool((y[2] == 0).all()) and bool(((r[2:4] - 1e3).abs() <= 1e-3).all())
        else:
            assert bool(torch.isinf(r[2:4]).all()) and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(q[2].float()).all())
