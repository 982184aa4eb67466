"""The RMS norm and the 8-bit entry points on the CPU: every check returns its status
before anything is enqueued (no call here reaches the HIP runtime), the workspace
sizes, and the binding's own refusals."""
import ctypes
import math

import pytest
import torch

import matrix_optimizers_amd as mo
from matrix_optimizers_amd import _binding as B
from matrix_optimizers_amd import fp8 as M8
from test_operators_abi import A, ALIAS, HUGE, INVALID, OK, UNSUPPORTED, WS_SMALL, size_of

FP8, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---- RMS norm ------------------------------------------------------------------------

def rms_fwd(X=A[0], ldx=0, res=A[1], ldr=0, w=A[2], H=A[3], ldh=0, Y=A[4], ldy=0, q=A[5], ldq=0, s=A[6], lds=0,
            rstd=A[7], rows=10, cols=300, dtype=1, eps=1e-6):
    return mo.load_library().rms_norm_forward(X, ldx, res, ldr, w, H, ldh, Y, ldy, q, ldq, s, lds, rstd, rows, cols,
                                              dtype, eps, None)


def rms_bwd(dY=A[0], lddy=0, H=A[1], ldh=0, w=A[2], rstd=A[3], dH=A[4], lddh=0, dX=A[5], lddx=0, dw=A[6], rows=10,
            cols=300, dtype=1, ws=A[8], have=HUGE):
    return mo.load_library().rms_norm_backward(dY, lddy, H, ldh, w, rstd, dH, lddh, dX, lddx, dw, rows, cols, dtype,
                                               ws, have, None)


def test_rms_norm_noops():
    assert rms_fwd(rows=0) == OK and rms_fwd(cols=0) == OK and rms_fwd(rows=0, X=None, Y=None, q=None, s=None) == OK
    assert rms_bwd(cols=0) == OK and rms_bwd(dX=None, dw=None, ws=None) == OK and rms_bwd(rows=0, dw=None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), INVALID), (dict(Y=None, q=None, s=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(res=None), INVALID),   # h is written only where there is a residual
    (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(ldx=299), INVALID), (dict(ldr=1), INVALID),
    (dict(ldh=1), INVALID), (dict(ldy=299), INVALID), (dict(ldq=299), INVALID), (dict(lds=2), INVALID),
    (dict(ldx=-300), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(cols=(1 << 24) + 1), UNSUPPORTED),
    (dict(rows=(1 << 32) + 1), UNSUPPORTED), (dict(ldx=(1 << 26) + 1), UNSUPPORTED),
    (dict(Y=A[0]), ALIAS), (dict(H=A[0]), ALIAS), (dict(H=A[1]), ALIAS), (dict(H=A[4] + 600), ALIAS),
    (dict(q=A[4] + 10), ALIAS), (dict(s=A[5] + 2999), ALIAS), (dict(rstd=A[2] + 4), ALIAS), (dict(s=A[7] + 39), ALIAS)])
def test_rms_norm_forward_refusals(kw, code):
    assert rms_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(H=None), INVALID), (dict(dY=None), INVALID), (dict(rstd=None), INVALID), (dict(rows=-1), INVALID),
    (dict(ldh=3), INVALID), (dict(lddy=3), INVALID), (dict(lddh=3), INVALID), (dict(lddx=3), INVALID),
    (dict(dtype=9), UNSUPPORTED), (dict(lddx=(1 << 26) + 1), UNSUPPORTED), (dict(dX=A[1]), ALIAS), (dict(dX=A[0]), ALIAS),
    (dict(dX=A[4]), ALIAS), (dict(dw=A[2]), ALIAS), (dict(dw=A[3] + 36), ALIAS), (dict(dw=A[5] + 64), ALIAS),
    (dict(ws=A[5]), ALIAS), (dict(ws=None), WS_SMALL), (dict(have=64), WS_SMALL)])
def test_rms_norm_backward_refusals(kw, code):
    assert rms_bwd(**kw) == code


def test_rms_norm_workspace():
    lib = mo.load_library()
    st, need = size_of(lib.rms_norm_workspace_bytes, 10, 300)
    assert st == OK and need >= 300 * 4 and rms_bwd(have=need - 1) == WS_SMALL
    assert size_of(lib.rms_norm_workspace_bytes, 0, 64) == (OK, 0)
    assert size_of(lib.rms_norm_workspace_bytes, -1, 64)[0] == INVALID
    assert lib.rms_norm_workspace_bytes(1, 1, None) == INVALID
    # a partial row per workgroup, not per row
    assert mo.rms_norm_workspace_bytes(1 << 20, 4096) < 32 << 20


# ---- casts -----------------------------------------------------------------------------

def quant(X=A[0], ldx=0, dtype=1, rows=10, cols=300, q=A[1], ldq=0, s=A[2], lds=0):
    return mo.load_library().fp8_quantize(X, ldx, dtype, rows, cols, q, ldq, s, lds, None)


def dequant(q=A[1], ldq=0, s=A[2], lds=0, rows=10, cols=300, X=A[0], ldx=0, dtype=1):
    return mo.load_library().fp8_dequantize(q, ldq, s, lds, rows, cols, X, ldx, dtype, None)


def weight(W=A[0], ldw=0, dtype=1, rows=200, cols=300, q=A[1], ldq=0, s=A[2], lds=0, qt=A[3], ldqt=0, st=A[4], ldst=0):
    return mo.load_library().fp8_quantize_weight(W, ldw, dtype, rows, cols, q, ldq, s, lds, qt, ldqt, st, ldst, None)


@pytest.mark.parametrize("call", [quant, dequant])
@pytest.mark.parametrize("kw,code", [
    (dict(X=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=-1), INVALID), (dict(ldx=299), INVALID), (dict(ldq=299), INVALID), (dict(lds=2), INVALID),
    (dict(lds=-3), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(rows=(1 << 32) + 1), UNSUPPORTED),
    (dict(cols=(1 << 24) + 1), UNSUPPORTED), (dict(ldq=(1 << 26) + 1), UNSUPPORTED), (dict(q=A[0] + 600), ALIAS),
    (dict(s=A[0] + 5999), ALIAS), (dict(rows=0, X=None, q=None, s=None), OK), (dict(cols=0), OK)])
def test_cast_refusals(call, kw, code):
    assert call(**kw) == code


def test_cast_reads_may_overlap():
    """Two read matrices may; a read and a written one may not."""
    assert quant(s=A[1] + 100) == ALIAS


@pytest.mark.parametrize("kw,code", [
    (dict(W=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(qt=None), INVALID),
    (dict(st=None), INVALID), (dict(q=None, s=None, qt=None, st=None), INVALID), (dict(rows=-1), INVALID),
    (dict(ldw=299), INVALID), (dict(ldq=299), INVALID), (dict(lds=2), INVALID), (dict(ldqt=199), INVALID),
    (dict(ldst=1), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(rows=(1 << 20) + 1), UNSUPPORTED),
    (dict(cols=(1 << 20) + 1), UNSUPPORTED), (dict(qt=A[1] + 8), ALIAS), (dict(st=A[2]), ALIAS), (dict(q=A[0]), ALIAS),
    (dict(rows=0), OK), (dict(cols=0, W=None), OK)])
def test_quantize_weight_refusals(kw, code):
    assert weight(**kw) == code


# ---- products --------------------------------------------------------------------------

def mat(q, s, rows, **kw):
    d = dict(ld_q=0, ld_scales=0, inc_scales=0, block_rows=1)
    d.update(kw)
    return B.MoFp8Matrix(q, s, rows, d["ld_q"], d["ld_scales"], d["inc_scales"], d["block_rows"])


def act(rows=500, **kw):
    return mat(kw.pop("q", A[0]), kw.pop("s", A[1]), rows, **kw)


def wei(rows=600, **kw):
    return mat(kw.pop("q", A[2]), kw.pop("s", A[3]), rows, block_rows=kw.pop("block_rows", 128), **kw)


def mm(a=None, b=None, dim=512, Y=A[4], ldy=0, dtype=1, ws=A[5], have=HUGE):
    return mo.load_library().fp8_matmul(a or act(), b or wei(), dim, Y, ldy, dtype, ws, have, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=act(q=None)), INVALID), (dict(a=act(s=None)), INVALID), (dict(b=wei(q=None)), INVALID),
    (dict(b=wei(s=None)), INVALID), (dict(Y=None), INVALID), (dict(dim=-1), INVALID), (dict(a=act(rows=-1)), INVALID),
    (dict(b=wei(rows=-5)), INVALID), (dict(a=act(ld_q=511)), INVALID), (dict(b=wei(ld_q=511)), INVALID),
    (dict(a=act(ld_scales=3)), INVALID), (dict(b=wei(ld_scales=3)), INVALID), (dict(ldy=599), INVALID),
    (dict(a=act(block_rows=0)), INVALID), (dict(a=act(block_rows=64)), INVALID), (dict(b=wei(block_rows=256)), INVALID),
    # by columns: the rows are 1 apart, the columns no less than the rows
    (dict(a=act(inc_scales=500)), INVALID), (dict(a=act(ld_scales=1, inc_scales=499)), INVALID),
    (dict(b=wei(ld_scales=1, inc_scales=4)), INVALID), (dict(a=act(ld_scales=1, inc_scales=-500)), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dim=(1 << 20) + 1), UNSUPPORTED), (dict(a=act(rows=(1 << 20) + 1)), UNSUPPORTED),
    (dict(b=wei(rows=(1 << 20) + 1)), UNSUPPORTED), (dict(a=act(ld_q=1 << 23)), UNSUPPORTED),
    (dict(b=wei(ld_q=1 << 23)), UNSUPPORTED), (dict(a=act(ld_scales=1 << 23)), UNSUPPORTED),
    (dict(ldy=(1 << 26) + 1), UNSUPPORTED), (dict(a=act(ld_scales=1, inc_scales=(1 << 26) + 1)), UNSUPPORTED),
    (dict(Y=A[0] + 100), ALIAS), (dict(Y=A[3] + 4), ALIAS), (dict(dtype=0, Y=A[2]), ALIAS),
    (dict(a=act(rows=3), Y=A[2] + 16), ALIAS), (dict(a=act(rows=3), Y=A[1] + 11), ALIAS),
    (dict(a=act(rows=0)), OK), (dict(b=wei(rows=0), Y=None), OK), (dict(a=act(rows=0, q=None, s=None), Y=None), OK)])
def test_matmul_refusals(kw, code):
    assert mm(**kw) == code


def test_matmul_null_operands():
    lib = mo.load_library()
    assert lib.fp8_matmul(None, wei(), 512, A[4], 0, 1, A[5], HUGE, None) == INVALID
    assert lib.fp8_matmul(act(), None, 512, A[4], 0, 1, A[5], HUGE, None) == INVALID
    out = ctypes.c_size_t(5)
    assert lib.fp8_matmul_workspace_bytes(None, wei(), 512, 1, out) == INVALID and out.value == 0
    assert lib.fp8_matmul_workspace_bytes(act(), wei(), 512, 1, None) == INVALID


def mm_bytes(a, b, dim, dtype=1):
    out = ctypes.c_size_t(0)
    assert mo.load_library().fp8_matmul_workspace_bytes(a, b, dim, dtype, out) == OK
    return out.value


def test_matmul_workspace():
    # parts along a long K of few tiles; none for a grid of whole rounds, a small product or no work
    long = act(1500), wei(1000), 16384
    need = mm_bytes(*long)
    assert need > 0 and mm(*long, have=need - 1) == WS_SMALL
    assert mm(*long, ws=None) == WS_SMALL
    assert mm(*long, ws=A[4] + 64) == ALIAS
    assert mm_bytes(act(4096), wei(4096), 4096) == 0
    for few in (1, 32):
        assert mm_bytes(act(few), wei(4096), 4096) == 0 and mm_bytes(act(few), wei(4096), 500) == 0
    for args in ((act(0), wei(), 512), (act(), wei(0), 512), (act(), wei(), 0)):
        assert mm_bytes(*args) == 0
    # for a bf16 result in 8 bits an unaligned operand is copied where that pays; for an fp32 result
    # it is converted as it is read
    assert 16384 * 4096 <= mm_bytes(act(16384, q=A[0] + 1), wei(16384), 4096) < 1.1 * 16384 * 4096
    assert mm_bytes(act(16384), wei(16384), 4000) >= 2 * 16384 * 4000
    assert mm_bytes(act(1500), wei(128), 4000) < 1500 * 4000
    assert mm_bytes(act(16384, q=A[0] + 1), wei(14336), 4096, dtype=0) < 16384 * 4096
    # scales that are not whole aligned dwords are copied
    assert mm_bytes(act(4096, s=A[1] + 1), wei(4096), 4096) >= 4096 * 32
    assert mm_bytes(act(4096, ld_scales=1, inc_scales=4096), wei(4096), 4096) >= 4096 * 32


def test_a_weights_scales_are_never_copied():
    """Whatever their strides and alignment: of 128 rows each they are read singly."""
    for kw in (dict(), dict(s=A[3] + 1), dict(ld_scales=33), dict(ld_scales=1, inc_scales=32), dict(ld_scales=1, inc_scales=99)):
        assert mm_bytes(act(4096), wei(4096, **kw), 4096) == 0


def wg(dY=A[0], ldy=0, yt=1, x="default", dim=512, G=A[4], ldg=0, gt=0, rows=600, acc=0, ws=A[5], have=HUGE):
    x = wei(500, block_rows=1) if x == "default" else x
    return mo.load_library().fp8_weight_grad(dY, ldy, yt, x, dim, G, ldg, gt, rows, acc, ws, have, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(dY=None), INVALID), (dict(G=None), INVALID), (dict(x=wei(500)), INVALID),
    (dict(x=wei(500, block_rows=1, q=None)), INVALID), (dict(x=wei(500, block_rows=1, s=None)), INVALID),
    (dict(x=wei(-1, block_rows=1)), INVALID), (dict(dim=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(ldy=599), INVALID), (dict(ldg=511), INVALID), (dict(x=wei(500, block_rows=1, ld_q=511)), INVALID),
    (dict(yt=2), UNSUPPORTED), (dict(gt=2), UNSUPPORTED), (dict(dim=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(x=wei((1 << 20) + 1, block_rows=1)), UNSUPPORTED),
    (dict(ldy=(1 << 26) + 1), UNSUPPORTED), (dict(G=A[0] + 64), ALIAS), (dict(G=A[2]), ALIAS), (dict(G=A[3] + 1), ALIAS),
    (dict(x=wei(16384, block_rows=1), ws=A[4]), ALIAS), (dict(x=wei(16384, block_rows=1), have=4096), WS_SMALL),
    (dict(x=wei(16384, block_rows=1), ws=None), WS_SMALL),
    (dict(rows=0), OK), (dict(dim=0, G=None), OK), (dict(x=wei(0, block_rows=1), acc=1, G=None), OK)])
def test_weight_grad_refusals(kw, code):
    assert wg(**kw) == code


def wg_bytes(dY=A[0], ldy=0, yt=1, x="default", dim=512, rows=600):
    out = ctypes.c_size_t(7)
    x = wei(500, block_rows=1) if x == "default" else x
    st = mo.load_library().fp8_weight_grad_workspace_bytes(dY, ldy, yt, x, dim, rows, out)
    return st, out.value


def test_weight_grad_workspace():
    big = dict(x=wei(16384, block_rows=1), dim=4096, rows=4096)
    assert wg_bytes(**big) == (OK, 0)                      # whole rounds of tiles, read in place
    st, need = wg_bytes(yt=0, **big)                       # three bf16 parts of dY and one of X, transposed
    assert st == OK and need >= (3 + 1) * 16384 * 4096 * 2
    assert wg_bytes(dY=A[0] + 2, **big)[1] >= 2 * 16384 * 4096 * 2
    assert wg_bytes(ldy=4097, **big)[1] >= 2 * 16384 * 4096 * 2
    assert wg_bytes() == (OK, 0)                           # a small one takes no workspace
    long = dict(x=wei(16384, block_rows=1))                # many are, of 3 x 2 to 8 tiles
    st, need = wg_bytes(**long)
    assert st == OK and need >= 2 * 600 * 512 * 4 and wg(have=need - 1, **long) == WS_SMALL
    for none in (dict(rows=0), dict(dim=0), dict(x=wei(0, block_rows=1))):
        assert wg_bytes(**none) == (OK, 0)
    assert wg_bytes(x=None)[0] == INVALID
    assert mo.load_library().fp8_weight_grad_workspace_bytes(A[0], 0, 1, wei(500, block_rows=1), 512, 600, None) == INVALID


# ---- the binding's checks ------------------------------------------------------------------

def host8(rows, cols, r=1):
    return torch.zeros((rows, cols)).to(FP8), torch.ones((-(-rows // r), -(-cols // 128))).to(SCALE)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 128)
    q, s = host8(4, 128)
    for call in (lambda: mo.rms_norm_forward(x), lambda: mo.rms_norm_quantize(x), lambda: mo.rms_norm_backward(x, x, x[:, 0]),
                 lambda: mo.fp8_quantize(x), lambda: mo.fp8_dequantize(q, s), lambda: mo.fp8_quantize_weight(x),
                 lambda: mo.fp8_matmul(q, s, q, s), lambda: mo.fp8_weight_grad(x, q, s, x.clone())):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_binding_operands():
    q, s = host8(300, 300)
    m = M8._operand(q, s, "A")
    assert (m.rows, m.ld_q, m.ld_scales, m.inc_scales, m.block_rows) == (300, 300, 3, 0, 1)
    m = M8._operand(*host8(300, 300, 128), "B")
    assert (m.rows, m.ld_scales, m.inc_scales, m.block_rows) == (300, 3, 0, 128)
    st = host8(300, 300, 128)[1].view(torch.uint8).t().view(SCALE)
    m = M8._operand(q, st, "B")
    assert (m.ld_scales, m.inc_scales, m.block_rows) == (1, 3, 128)
    cols = s.view(torch.uint8).t().contiguous().t().view(SCALE)
    m = M8._operand(q, cols, "A")
    assert (m.ld_scales, m.inc_scales, m.block_rows) == (1, 300, 1)
    for bad in (s[:, :2], s[:200], host8(300, 300, 64)[1]):
        with pytest.raises(ValueError):
            M8._operand(q, bad, "A")
    with pytest.raises(ValueError):
        M8._operand(q, host8(300, 300, 128)[1], "q", square=False)
    with pytest.raises(TypeError):
        M8._operand(q.float(), s, "A")
    with pytest.raises(TypeError):
        M8._operand(q, s.float(), "A")
    with pytest.raises(TypeError):
        M8._operand(q.view(torch.uint8), s, "A")
    with pytest.raises(ValueError, match="same columns"):
        M8._matmul_args(q, s, *host8(300, 200))
    with pytest.raises(TypeError):
        mo.fp8_matmul_workspace_bytes(q, s, q, s, dtype=torch.float16)
    assert mo.fp8_matmul_workspace_bytes(q, s, q, s) == 0 and mo.fp8_matmul_workspace_bytes(*host8(1500, 16384), *host8(1000, 16384)) > 0
    assert mo.fp8_weight_grad_workspace_bytes(torch.zeros(64, 7), *host8(64, 300)) == 0
    assert mo.fp8_weight_grad_workspace_bytes(torch.zeros(16384, 7), *host8(16384, 300)) > 0
    with pytest.raises(ValueError):
        mo.fp8_weight_grad_workspace_bytes(torch.zeros(299, 7), q, s)
    with pytest.raises(TypeError):
        mo.fp8_weight_grad_workspace_bytes(torch.zeros(300, 7, dtype=torch.float16), q, s)
