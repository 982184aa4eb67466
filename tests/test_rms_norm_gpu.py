"""The RMS norm's kernels against their 64-bit formulas."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
import operators_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (3, 7), (5, 64), (33, 100), (130, 128), (7, 200), (65, 512), (9, 520), (257, 1000), (70, 1024),
          (1, 4096), (300, 4096), (19, 4104), (21, 8200), (5, 16384), (3, 16385), (2, 20000), (4, 33000)]


def inputs(rows, cols, dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * rows + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda") * scale
    x *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
    res = torch.randn((rows, cols), generator=g, device="cuda") * scale
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    return x.to(dtype), res.to(dtype), w


def check8(q, s, y, rel, what):
    """q and s hold y, which the kernel has to a relative `rel`."""
    top = F.row_amax(y)
    b = F.codes(s).double()
    assert bool(((b >= F.bytes_of(top * (1 - rel))) & (b <= F.bytes_of(top * (1 + rel)))).all()), what
    sc = F.spread(torch.exp2(b - 127), *y.shape)
    v = (y / sc).abs()
    half = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 4)
    R.check(q.double() * sc, y, (half + rel * v) * (1 + 2.0 ** -3) * sc, what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    x, res, w = inputs(rows, cols, dtype)
    rel = F.rms_r_bound(cols) + 3 * R.U
    for residual in (None, res):
        for weight in (w, None):
            Y, h, rstd = mo.rms_norm_forward(x, weight, residual=residual)
            if residual is None:
                assert h is x
            else:
                assert torch.equal(h, (x.float() + res.float()).to(dtype))
            y, r = F.rms(h, weight, 1e-6)
            R.check(rstd, r, F.rms_r_bound(cols) * r, "rstd")
            R.check(Y, y, (rel + R.ut(dtype)) * y.abs(), "Y")
            q, s, h2, rstd2 = mo.rms_norm_quantize(x, weight, residual=residual)
            assert torch.equal(h2, h) and torch.equal(rstd2, rstd)
            check8(q, s, y, rel, "q")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, dtype):
    h, dH, w = inputs(rows, cols, dtype, seed=1)
    dY = inputs(rows, cols, dtype, seed=2)[1]
    r = F.rms(h, None, 1e-6)[1].float()
    for weight in (w, None):
        for d in (dH, None):
            dX, dw = mo.rms_norm_backward(dY, h, r, weight, dH=d)
            (want, wantw), (b, bw) = F.rms_grad(dY, h, r, weight, d)
            R.check(dX, want, b, "dX")
            R.check(dw, wantw, bw, "dw")
    only, none = mo.rms_norm_backward(dY, h, r, w, need_dweight=False)
    assert none is None and torch.equal(only, mo.rms_norm_backward(dY, h, r, w)[0])
    none, only = mo.rms_norm_backward(dY, h, r, w, need_dX=False)
    assert none is None and torch.equal(only, mo.rms_norm_backward(dY, h, r, w)[1])


def test_gradient_by_differences():
    """dX and dw against central differences of the 64-bit formula.  With steps of 2^-12 the
    differences are off by at most 2^-25 of third derivatives (below 30 here)."""
    rows, cols, t = 3, 40, 2.0 ** -12
    x, dY, w = (a.double() for a in inputs(rows, cols, F32, seed=5))
    f = lambda x, w: float((F.rms(x, w, 1e-6)[0] * dY).sum())
    _, _, r = mo.rms_norm_forward(x.float(), w.float())
    dX, dw = mo.rms_norm_backward(dY.float(), x.float(), r, w.float())
    for i in range(rows):
        for j in range(cols):
            e = torch.zeros_like(x)
            e[i, j] = t
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * t) - float(dX[i, j])) < 2e-5
    for j in range(cols):
        e = torch.zeros_like(w)
        e[j] = t
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * t) - float(dw[j])) < 2e-5


def test_strides_and_what_lies_around():
    """Rows at odd strides and addresses; what lies between and behind them stays."""
    rows, cols, ld = 21, 300, 333
    x, res, w = inputs(rows, cols, BF16)

    def inside(t, fill=7.0):
        big = torch.full((rows + 1, ld), fill, device="cuda").to(t.dtype)
        big[:rows, 5:5 + cols] = t
        return big, big[:rows, 5:5 + cols]
    bx, vx = inside(x)
    br, vr = inside(res)
    want = mo.rms_norm_forward(x, w, residual=res)
    wantq = mo.rms_norm_quantize(x, w, residual=res)
    by, vy = inside(torch.zeros_like(x))
    bh, vh = inside(torch.zeros_like(x))
    mo.rms_norm_forward(vx, w, residual=vr, out=vy, h=vh)
    assert torch.equal(vy, want[0]) and torch.equal(vh, want[1])
    bq = torch.full((rows + 1, ld), 9, dtype=torch.uint8, device="cuda").view(F.FP8)
    bs = torch.full((rows + 1, 11), 9, dtype=torch.uint8, device="cuda").view(F.SCALE)
    mo.rms_norm_quantize(vx, w, residual=vr, q=bq[:rows, 5:5 + cols], scales=bs[:rows, 3:6], h=vh)
    assert torch.equal(F.codes(bq)[:rows, 5:5 + cols], F.codes(wantq[0]))
    assert torch.equal(F.codes(bs)[:rows, 3:6], F.codes(wantq[1]))
    bd, vd = inside(torch.zeros_like(x))
    mo.rms_norm_backward(vr, vx, want[2], w, dH=vr, dX=vd)
    assert torch.equal(vd, mo.rms_norm_backward(res, x, want[2], w, dH=res)[0])
    for big in (by, bh, bd):
        big = big.clone()
        big[:rows, 5:5 + cols] = 7
        assert bool((big == 7).all())
    for big, lo, hi in ((F.codes(bq), 5, 5 + cols), (F.codes(bs), 3, 6)):
        big = big.clone()
        big[:rows, lo:hi] = 9
        assert bool((big == 9).all())


def test_rows_of_zeros_and_bad_values():
    """A row of zeros has y = 0 and rstd eps^-1/2; a NaN or an infinity stays in its row."""
    x, res, w = inputs(6, 512, BF16)
    x[1] = 0
    x[3, 17] = float("nan")
    x[4, 200] = float("inf")
    Y, h, rstd = mo.rms_norm_forward(x, w)
    q, s, _, _ = mo.rms_norm_quantize(x, w)
    assert float(rstd[1]) == pytest.approx(1e3, rel=1e-6) and bool((Y[1] == 0).all())
    assert bool((F.codes(s)[1] == 0).all()) and bool((q[1].float() == 0).all())
    assert bool(torch.isnan(Y[3]).all()) and bool(torch.isnan(q[3].float()).all())
    good = [0, 1, 2, 5]
    Z, _, r2 = mo.rms_norm_forward(x[good], w)
    assert torch.equal(Y[good], Z) and torch.equal(rstd[good], r2)
    assert not bool(torch.isfinite(Y[4, 200])) and bool((Y[4, :200] == 0).all())   # over an infinite norm


def test_empty():
    e = torch.empty((0, 64), device="cuda")
    Y, h, r = mo.rms_norm_forward(e)
    assert Y.shape == (0, 64) and r.shape == (0,)
    q, s, _, _ = mo.rms_norm_quantize(e)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    dX, dw = mo.rms_norm_backward(e, e, r)
    assert dX.shape == (0, 64) and bool((dw == 0).all())
    Y, _, r = mo.rms_norm_forward(torch.empty((3, 0), device="cuda"))
    assert Y.shape == (3, 0) and bool(torch.isnan(r).all())
