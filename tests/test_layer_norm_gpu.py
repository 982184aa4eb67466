"""Layer norm forward and backward against the 64-bit form, within the bounds
derived in operators_ref.py."""
import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand, strided, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# one row to several workgroups' worth; teams of 8 threads up to whole workgroups with one,
# two and four chunks per thread, and rows too long for registers
SHAPES = [(1, 1), (1, 8), (3, 7), (33, 64), (257, 65), (40, 300), (513, 512), (6, 520), (2049, 1000), (5, 4096),
          (9, 8192), (3, 8193), (4, 16384), (3, 16385), (2, 20001), (2, 32768), (3, 32769), (2, 70001)]


def case(rows, cols, dtype, affine, pad):
    g = gen(rows * 31 + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda") * 2 + 3 * torch.randn((rows, 1), generator=g, device="cuda")
    X, _ = strided(x.to(dtype), pad, 1 if pad else 0)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    b = torch.randn(cols, generator=g, device="cuda")
    # slices of a packed tail start at any element
    tail = torch.cat([torch.zeros(3, device="cuda"), w, b])
    return g, X, tail[3:3 + cols] if affine else None, tail[3 + cols:] if affine else None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("affine,pad", [(True, 0), (False, 5)])
def test_forward(gpu, dtype, rows, cols, affine, pad):
    _, X, w, b = case(rows, cols, dtype, affine, pad)
    out, buf = strided(torch.zeros(rows, cols, device="cuda", dtype=dtype), pad, pad // 2)
    Y, mean, rstd = mo.layer_norm_forward(X, w, b, eps=1e-5, out=out)
    torch.cuda.synchronize()
    eps = torch.tensor(1e-5, dtype=F32).double().item()
    y, mu, r = R.norm(X, w, b, eps)
    by, bmu, br = R.norm_bounds(X, w, b, eps, dtype)
    R.check(Y, y, by, "Y")
    R.check(mean, mu, bmu, "mean")
    R.check(rstd, r, br, "rstd")
    assert untouched(out, buf)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("affine,pad", [(True, 0), (False, 5)])
def test_backward(gpu, dtype, rows, cols, affine, pad):
    g, X, w, b = case(rows, cols, dtype, affine, pad)
    _, mean, rstd = mo.layer_norm_forward(X, w, b)
    dY, _ = strided(rand(g, (rows, cols), dtype), pad, pad // 3)
    dX, buf = strided(torch.zeros(rows, cols, device="cuda", dtype=dtype), pad, pad // 2)
    tail = torch.full((2 * cols + 5,), 77.0, device="cuda")
    dw, db = tail[1:1 + cols], tail[3 + cols:3 + 2 * cols]
    mo.layer_norm_backward(dY, X, mean, rstd, w, dX=dX, dweight=dw, dbias=db)
    torch.cuda.synchronize()
    (dx, gw, gb), (bx, bw, bb) = R.norm_grad(dY, X, mean, rstd, w)
    R.check(dX, dx, bx, "dX")
    R.check(dw, gw, bw, "dweight")
    R.check(db, gb, bb, "dbias")
    assert untouched(dX, buf)
    assert bool((tail[[0, 1 + cols, 2 + cols, 3 + 2 * cols, 4 + 2 * cols]] == 77).all())


@pytest.mark.parametrize("cols", [48, 1000, 20000])
def test_parts_of_the_backward_pass(gpu, cols):
    """Each gradient alone equals, bit for bit, the one from the call for all three."""
    g, X, w, b = case(70, cols, BF, True, 0)
    _, mean, rstd = mo.layer_norm_forward(X, w, b)
    dY = rand(g, (70, cols), BF)
    full = mo.layer_norm_backward(dY, X, mean, rstd, w)
    for k, name in enumerate(("dX", "dweight", "dbias")):
        need = {f"need_{n}": n == name for n in ("dX", "dweight", "dbias")}
        got = mo.layer_norm_backward(dY, X, mean, rstd, w, **need)
        torch.cuda.synchronize()
        assert [x is not None for x in got] == [i == k for i in range(3)]
        assert torch.equal(got[k], full[k])


def test_large_offset_and_outlier(gpu):
    """Rows whose mean is 1000 times their spread, and with one entry of 1e4: the
    variance is taken about the finished mean."""
    g = gen(1)
    x = torch.randn(8, 4096, generator=g, device="cuda")
    x[:4] += 1000
    x[4:, 17] = 1e4
    y, mean, rstd = mo.layer_norm_forward(x)
    torch.cuda.synchronize()
    eps = torch.tensor(1e-5, dtype=F32).double().item()
    want = R.norm(x, None, None, eps)
    bounds = R.norm_bounds(x, None, None, eps, F32)
    for a, b, c, n in zip((y, mean, rstd), want, bounds, ("Y", "mean", "rstd")):
        R.check(a, b, c, n)


def test_constant_rows_and_non_finite_rows_stay_apart(gpu):
    x = torch.randn(6, 100, generator=gen(2), device="cuda")
    x[1] = 3.0                     # zero variance: y = b
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    w, b = torch.ones(100, device="cuda"), torch.full((100,), 0.25, device="cuda")
    y, mean, rstd = mo.layer_norm_forward(x, w, b)
    torch.cuda.synchronize()
    assert bool((y[1] == 0.25).all())
    assert bool(torch.isfinite(y[[0, 1, 2, 5]]).all()) and bool(torch.isnan(y[3]).all())
    assert not bool(torch.isfinite(y[4]).all())


def test_empty(gpu):
    x = torch.zeros(0, 12, device="cuda")
    y, mean, rstd = mo.layer_norm_forward(x)
    dx, dw, db = mo.layer_norm_backward(x, x, mean, rstd, dweight=torch.ones(12, device="cuda"),
                                        dbias=torch.ones(12, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == dx.shape == (0, 12) and bool((dw == 0).all()) and bool((db == 0).all())


def test_gradient_by_differences(gpu):
    """The kernels' gradients against central differences of the 64-bit forward: a
    step of 1e-5 leaves a truncation error below 1e-8 of the derivative here; the
    gradients' own fp32 error, 1e-6 of the sum of the products' magnitudes."""
    g = gen(4)
    X, dY = rand(g, (5, 200), F32), rand(g, (5, 200), F32)
    w, b = rand(g, (200,), F32), rand(g, (200,), F32)
    _, mean, rstd = mo.layer_norm_forward(X, w, b)
    dx, dw, db = mo.layer_norm_backward(dY, X, mean, rstd, w)
    torch.cuda.synchronize()
    eps = torch.tensor(1e-5, dtype=F32).double().item()
    f = lambda x, ww, bb: (R.norm(x, ww, bb, eps)[0] * dY.double()).sum()
    for grad, k in ((dx, 0), (dw, 1), (db, 2)):
        args = [X.double(), w.double(), b.double()]
        v = rand(g, grad.shape, F32).double()
        hi, lo = list(args), list(args)
        hi[k], lo[k] = args[k] + 1e-5 * v, args[k] - 1e-5 * v
        num = float((f(*hi) - f(*lo)) / 2e-5)
        assert abs(float((grad.double() * v).sum()) - num) <= 1e-6 * float((grad.double() * v).abs().sum()) + 1e-6
