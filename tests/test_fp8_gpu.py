"""Matrices in 8 bits: casts, products and the weight's gradient against 64-bit formulas."""
import pytest
import torch

import fp8_ref as F
import matrix_optimizers_amd as mo
import operators_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) & 0x7FFFFFFF)


def matrix(rows, cols, dtype, *seed, spread=1.0):
    g = gen(rows, cols, *seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn((rows, 1), generator=g, device="cuda"))).to(dtype)


def same8(got, want):
    """Equal values, NaN where NaN is."""
    got = got.double()
    assert bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


CASTS = [(1, 1), (2, 127), (3, 128), (5, 129), (64, 200), (33, 1000), (1, 4096), (130, 2048), (257, 2049), (7, 28672),
         (1000, 16)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", CASTS)
def test_quantize(rows, cols, dtype):
    x = matrix(rows, cols, dtype, 1, spread=8.0)
    if rows > 2:
        x[1] = 0
    q, s = mo.fp8_quantize(x)
    wq, wb = F.quantize(x)
    assert q.dtype == F.FP8 and s.dtype == F.SCALE and s.shape == (rows, F.blocks(cols))
    assert torch.equal(F.codes(s).double(), wb)
    same8(q, wq)
    for out in (BF16, F32):
        y = mo.fp8_dequantize(q, s, dtype=out)
        assert y.dtype == out and torch.equal(y.double(), F.value(q, s))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", CASTS)
def test_quantize_weight(rows, cols, dtype):
    x = matrix(rows, cols, dtype, 2, spread=0.3)
    q, s, qt, st = mo.fp8_quantize_weight(x)
    wq, wb = F.quantize(x, 128)
    assert torch.equal(F.codes(s).double(), wb)
    same8(q, wq)
    assert torch.equal(F.codes(qt), F.codes(q).t()) and torch.equal(F.codes(st), F.codes(s).t())
    q2, s2, none, none2 = mo.fp8_quantize_weight(x, need_t=False)
    assert none is None and none2 is None and torch.equal(F.codes(q2), F.codes(q)) and torch.equal(F.codes(s2), F.codes(s))


def test_borders():
    """Every e4m3 number, every middle of two and their neighbours, in blocks whose largest is 448;
    blocks whose largest is on, just under and just over a border; subnormal and huge blocks."""
    grid = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(F.FP8).float()
    mid = (grid[1:] + grid[:-1]) / 2
    up = torch.nextafter(mid, torch.full_like(mid, 1e9))
    down = torch.nextafter(mid, torch.full_like(mid, -1e9))
    v = torch.cat([grid, -grid, mid, -mid, up, -up, down, -down])
    x = torch.full((-(-v.numel() // 127), 128), 0.0, device="cuda")
    x[:, 127] = 448
    for i in range(x.shape[0]):
        part = v[127 * i:127 * i + 127]
        x[i, :part.numel()] = part
    for shift in (0, 40, -40, -126):
        y = x * 2.0 ** shift
        q, s = mo.fp8_quantize(y)
        wq, wb = F.quantize(y)
        assert torch.equal(F.codes(s).double(), wb)
        same8(q, wq)
    edges = []
    for e in (-149, -140, -127, -119, -118, -9, -8, 0, 1, 9, 100, 119, 120):
        t = torch.tensor(1.75, device="cuda") * 2.0 ** (e + 0.0)
        edges += [t, torch.nextafter(t, torch.tensor(0.0, device="cuda")),
                  torch.nextafter(t, torch.tensor(float("inf"), device="cuda"))]
    edges += [torch.tensor(torch.finfo(F32).max, device="cuda"), torch.tensor(2.0 ** -149, device="cuda")]
    x = torch.zeros((len(edges), 128), device="cuda")
    x[:, 5] = torch.stack(edges)
    x[:, 6] = -x[:, 5] / 3
    q, s = mo.fp8_quantize(x)
    wq, wb = F.quantize(x)
    assert torch.equal(F.codes(s).double(), wb)
    same8(q, wq)


def test_bad_values_stay_alone():
    x = matrix(4, 300, BF16, 3)
    want = F.quantize(x)
    x2 = x.clone()
    x2[1, 5], x2[2, 130], x2[3, 299] = float("nan"), float("inf"), -float("inf")
    q, s = mo.fp8_quantize(x2)
    wq, wb = F.quantize(x2)
    assert torch.equal(F.codes(s).double(), wb)
    same8(q, wq)
    bad = torch.isnan(q.float())
    assert int(bad.sum()) == 3 and bool(bad[1, 5] & bad[2, 130] & bad[3, 299])
    assert torch.equal(wb[0], want[1][0])
    # a scale of 255 is NaN for its block
    F.codes(s)[0, 1] = 255
    y = mo.fp8_dequantize(q, s)
    assert bool(torch.isnan(y[0, 128:256]).all()) and bool(torch.isfinite(y[0, :128]).all())


@pytest.mark.parametrize("cast", ["rows", "weight", "back"])
def test_cast_strides(cast):
    rows, cols, ld = 37, 300, 411
    big = torch.zeros((rows + 1, ld), device="cuda", dtype=BF16)
    x = big[:rows, 3:3 + cols]
    x.copy_(matrix(rows, cols, BF16, 4))
    bytes_ = lambda r, c: torch.full((r, c), 9, dtype=torch.uint8, device="cuda")
    bq, bs = bytes_(rows + 1, ld), bytes_(rows + 1, 8)
    q, s = bq.view(F.FP8)[:rows, 5:5 + cols], bs.view(F.SCALE)[:rows, 1:4]
    if cast == "weight":
        s = s[:1]
        bqt, bst = bytes_(cols + 1, 50), bytes_(4, 3)
        qt, st = bqt.view(F.FP8)[:cols, 1:1 + rows], bst.view(F.SCALE)[:3, 1:2]
        mo.fp8_quantize_weight(x, q=q, scales=s, qt=qt, scales_t=st)
        want = mo.fp8_quantize_weight(x.contiguous())
        for a, b in zip((q, s, qt, st), want):
            assert torch.equal(F.codes(a), F.codes(b))
        bqt[:cols, 1:1 + rows] = 9
        bst[:3, 1:2] = 9
        assert bool((bqt == 9).all()) and bool((bst == 9).all())
        bs[:1, 1:4] = 9
    else:
        mo.fp8_quantize(x, q=q, scales=s)
        want = mo.fp8_quantize(x.contiguous())
        assert torch.equal(F.codes(q), F.codes(want[0])) and torch.equal(F.codes(s), F.codes(want[1]))
        if cast == "back":
            out = torch.full((rows + 1, ld), 7.0, device="cuda")
            mo.fp8_dequantize(q, s, out=out[:rows, 9:9 + cols])
            assert torch.equal(out[:rows, 9:9 + cols].double(), F.value(*want))
            out[:rows, 9:9 + cols] = 7
            assert bool((out == 7).all())
        bs[:rows, 1:4] = 9
    bq[:rows, 5:5 + cols] = 9
    assert bool((bq == 9).all()) and bool((bs == 9).all())


# ---- products ------------------------------------------------------------------------

PRODUCTS = [(1, 1, 1), (1, 16, 128), (3, 5, 127), (2, 300, 129), (8, 512, 512), (17, 257, 640), (64, 256, 1024),
            (65, 255, 1000), (130, 700, 384), (256, 256, 256), (257, 1025, 512), (300, 511, 2048), (40, 2001, 4096),
            (1021, 700, 1536), (5, 8192, 8192), (700, 900, 16)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(m, n, k, dtype):
    A, sa = mo.fp8_quantize(matrix(m, k, F32, 5))
    B, sb, _, _ = mo.fp8_quantize_weight(matrix(n, k, F32, 6, spread=0.3))
    Y = mo.fp8_matmul(A, sa, B, sb, dtype=dtype)
    want, bound = F.matmul(A, sa, B, sb, 1, 128, dtype)
    assert Y.dtype == dtype
    R.check(Y, want, bound, "Y")
    off = float((Y.double() - want).norm() / want.norm())
    assert off <= (R.ut(dtype) if dtype == BF16 else 2e-6), off
    # the scales of B by rows, and as the two sides change places
    B1, sb1 = mo.fp8_quantize(matrix(n, k, F32, 6, spread=0.3))
    want, bound = F.matmul(A, sa, B1, sb1, 1, 1, dtype)
    R.check(mo.fp8_matmul(A, sa, B1, sb1, dtype=dtype), want, bound, "Y by rows")
    want, bound = F.matmul(B, sb, A, sa, 128, 1, dtype)
    R.check(mo.fp8_matmul(B, sb, A, sa, dtype=dtype), want, bound, "Y^T")


def test_matmul_scales():
    """Scales far apart along K and between rows meet the right blocks."""
    m, n, k = 300, 520, 2048
    A, sa = mo.fp8_quantize(matrix(m, k, F32, 7))
    B, sb = mo.fp8_quantize(matrix(n, k, F32, 8))
    g = gen(9)
    for s in (sa, sb):
        F.codes(s).copy_(torch.randint(107, 147, s.shape, generator=g, device="cuda"))
    for dtype in (BF16, F32):
        want, bound = F.matmul(A, sa, B, sb, 1, 1, dtype)
        R.check(mo.fp8_matmul(A, sa, B, sb, dtype=dtype), want, bound, str(dtype))


@pytest.mark.parametrize("m,n,k", [(4200, 4100, 128), (4200, 4100, 256), (4100, 4200, 384), (8192, 4096, 640),
                                   (4133, 5001, 1100), (300, 700, 8320), (130, 300, 16640), (4352, 4352, 8704)])
def test_matmul_many_tiles(m, n, k):
    """More tiles than CUs (one workgroup multiplies several, of one to many stages), K that is split, and
    more stages than one read of a weight's scales holds; each block's scale its own."""
    A, sa = mo.fp8_quantize(matrix(m, k, F32, 40))
    B, sb, _, _ = mo.fp8_quantize_weight(matrix(n, k, F32, 41, spread=0.3))
    g = gen(42, m, n, k)
    for s in (sa, sb):
        F.codes(s).copy_(torch.randint(122, 132, s.shape, generator=g, device="cuda"))
    for dtype in (BF16, F32):
        want, bound = F.matmul(A, sa, B, sb, 1, 128, dtype)
        Y = mo.fp8_matmul(A, sa, B, sb, dtype=dtype)
        R.check(Y, want, bound, str(dtype))
        off = float((Y.double() - want).norm() / want.norm())
        assert off <= (R.ut(dtype) if dtype == BF16 else 2e-6), off
    B1, sb1 = mo.fp8_quantize(matrix(n, k, F32, 41, spread=0.3))
    F.codes(sb1).copy_(torch.randint(122, 132, sb1.shape, generator=g, device="cuda"))
    want, bound = F.matmul(A, sa, B1, sb1, 1, 1, BF16)
    R.check(mo.fp8_matmul(A, sa, B1, sb1), want, bound, "by rows")


@pytest.mark.parametrize("k", [512, 500])
def test_matmul_strides(k):
    """Odd strides and addresses.  Where they change how the operands are read, a bf16 result comes from other
    MFMAs, so it is held to the formula; an fp32 result comes from the same ones either way."""
    m, n = 70, 300
    A, sa = mo.fp8_quantize(matrix(m, k, F32, 10))
    B, sb, _, _ = mo.fp8_quantize_weight(matrix(n, k, F32, 11))
    for dtype in (BF16, F32):
        want = mo.fp8_matmul(A, sa, B, sb, dtype=dtype)

        def odd(t, pad, at):
            big = torch.full((t.shape[0] + 1, t.shape[1] + pad), 0x7F, dtype=torch.uint8, device="cuda")
            v = big[:t.shape[0], at:at + t.shape[1]]
            v.copy_(F.codes(t))
            return v.view(t.dtype)
        big = torch.full((m + 1, n + 7), 7.0, device="cuda", dtype=dtype)
        got = mo.fp8_matmul(odd(A, 5, 3), odd(sa, 3, 1), odd(B, 9, 1), odd(sb, 6, 2), out=big[:m, 3:3 + n])
        R.check(got, *F.matmul(A, sa, B, sb, 1, 128, dtype), "odd strides")
        assert dtype == BF16 or torch.equal(got, want)
        big[:m, 3:3 + n] = 7
        assert bool((big == 7).all())


@pytest.mark.parametrize("m,n,k", [(70, 300, 512), (300, 1000, 1280), (33, 129, 300)])
def test_matmul_scales_by_columns(m, n, k):
    """Scales that are a transposed view: the same result, bit by bit."""
    A, sa = mo.fp8_quantize(matrix(m, k, F32, 30, spread=3.0))
    B, sb, Bt, sbt = mo.fp8_quantize_weight(matrix(n, k, F32, 31, spread=0.3))
    for dtype in (BF16, F32):
        want = mo.fp8_matmul(A, sa, B, sb, dtype=dtype)
        assert torch.equal(mo.fp8_matmul(A, sa, B, sbt.t(), dtype=dtype), want)
        cols = F.codes(sa).t().contiguous().view(F.SCALE).t()
        assert torch.equal(mo.fp8_matmul(A, cols, B, sbt.t(), dtype=dtype), want)
        assert torch.equal(mo.fp8_matmul(B, sbt.t(), A, cols, dtype=dtype), mo.fp8_matmul(B, sb, A, sa, dtype=dtype))
    dY = matrix(m, 200, BF16, 32)
    G = torch.empty((200, k), device="cuda")
    assert torch.equal(mo.fp8_weight_grad(dY, A, cols, G).clone(), mo.fp8_weight_grad(dY, A, sa, G))


def test_matmul_bad_values():
    """NaN in an element or a scale reaches its row and column alone."""
    A, sa = mo.fp8_quantize(matrix(70, 512, F32, 12))
    B, sb = mo.fp8_quantize(matrix(300, 512, F32, 13))
    F.codes(A)[5, 77] = 0x7F
    F.codes(sb)[9, 2] = 255
    for dtype in (BF16, F32):
        Y = mo.fp8_matmul(A, sa, B, sb, dtype=dtype)
        bad = torch.isnan(Y)
        want = torch.zeros_like(bad)
        want[5] = True
        want[:, 9] = True
        assert torch.equal(bad, want)


def test_matmul_empty():
    E = torch.empty
    def mat(m, k):
        return E((m, k), device="cuda").to(F.FP8), E((m, F.blocks(k)), device="cuda").to(F.SCALE)
    for dtype in (BF16, F32):
        assert mo.fp8_matmul(*mat(0, 256), *mat(5, 256), dtype=dtype).shape == (0, 5)
        assert mo.fp8_matmul(*mat(5, 256), *mat(0, 256), dtype=dtype).shape == (5, 0)
        assert bool((mo.fp8_matmul(*mat(3, 0), *mat(5, 0), dtype=dtype) == 0).all())


WGRADS = [(1, 1, 1), (1, 300, 128), (3, 5, 127), (64, 256, 256), (65, 257, 129), (200, 70, 1000), (257, 1000, 700),
          (700, 33, 16), (1021, 256, 512), (2048, 130, 300), (4096, 256, 256)]


@pytest.mark.parametrize("ydtype", [BF16, F32])
@pytest.mark.parametrize("gdtype", [BF16, F32])
@pytest.mark.parametrize("t,n,k", WGRADS)
def test_weight_grad(t, n, k, ydtype, gdtype):
    q, s = mo.fp8_quantize(matrix(t, k, F32, 14))
    dY = matrix(t, n, ydtype, 15)
    G = torch.full((n, k), float("nan"), device="cuda", dtype=gdtype)
    want, bound = F.wgrad(dY, q, s, gdtype)
    assert mo.fp8_weight_grad(dY, q, s, G) is G
    R.check(G, want, bound, "G")
    if gdtype == F32:
        assert float((G.double() - want).norm() / want.norm()) <= 2e-6
    old = matrix(n, k, gdtype, 16)
    G = old.clone()
    want, bound = F.wgrad(dY, q, s, gdtype, old)
    R.check(mo.fp8_weight_grad(dY, q, s, G, accumulate=True), want, bound, "G added")


@pytest.mark.parametrize("t,n,k,ydtype", [(64, 4200, 4100, BF16), (200, 4100, 4352, F32), (2048, 4400, 4400, BF16),
                                          (1030, 5001, 4133, F32)])
def test_weight_grad_many_tiles(t, n, k, ydtype):
    q, s = mo.fp8_quantize(matrix(t, k, F32, 43))
    dY = matrix(t, n, ydtype, 44)
    G = torch.full((n, k), float("nan"), device="cuda")
    want, bound = F.wgrad(dY, q, s, F32)
    R.check(mo.fp8_weight_grad(dY, q, s, G), want, bound, "G")
    assert float((G.double() - want).norm() / want.norm()) <= 2e-6
    G = torch.empty((n, k), device="cuda", dtype=BF16)
    want, bound = F.wgrad(dY, q, s, BF16)
    R.check(mo.fp8_weight_grad(dY, q, s, G), want, bound, "G in bf16")


@pytest.mark.parametrize("t,n,k", [(70, 136, 272), (129, 256, 256), (33, 33, 33)])
def test_weight_grad_bad_values(t, n, k):
    """Infinities and NaN reach the sums they are in and no others, from the last token too."""
    q, s = mo.fp8_quantize(matrix(t, k, F32, 45))
    dY = matrix(t, n, BF16, 46)
    dY[t - 1, 3] = float("inf")
    dY[5, 7] = float("nan")
    F.codes(q)[t - 1, 9] = 0x7F
    F.codes(s)[2, 0] = 255
    F.codes(q)[2, 30:] = 0x38
    x = F.value(q, s)
    want = dY.double().t() @ x
    for dt in (BF16, F32):
        G = mo.fp8_weight_grad(dY, q, s, torch.empty((n, k), device="cuda", dtype=dt)).double()
        assert torch.equal(torch.isnan(G), torch.isnan(want))
        assert torch.equal(G[torch.isinf(want)], want[torch.isinf(want)])
        assert torch.equal(torch.isinf(G), torch.isinf(want))


def test_weight_grad_scales():
    """Tokens' scales far apart, and those of 0 (2^-127)."""
    t, n, k = 300, 264, 528
    q, s = mo.fp8_quantize(matrix(t, k, F32, 47))
    g = gen(48)
    F.codes(s).copy_(torch.randint(107, 147, s.shape, generator=g, device="cuda"))
    F.codes(s)[::7] = 0
    for dY in (matrix(t, n, BF16, 49), matrix(t, n, F32, 49)):
        want, bound = F.wgrad(dY, q, s, F32)
        R.check(mo.fp8_weight_grad(dY, q, s, torch.empty((n, k), device="cuda")), want, bound, "G")


def test_weight_grad_by_differences():
    """Against differences of the loss sum(dY * (X W^T)), which is linear in W."""
    t, n, k = 9, 5, 140
    q, s = mo.fp8_quantize(matrix(t, k, F32, 17))
    dY = matrix(t, n, F32, 18)
    G = mo.fp8_weight_grad(dY, q, s, torch.empty((n, k), device="cuda"))
    x, W = F.value(q, s), matrix(n, k, F32, 19).double()
    f = lambda W: float((dY.double() * (x @ W.t())).sum())
    for i, j in ((0, 0), (1, 3), (4, 139), (2, 128), (3, 127)):
        e = torch.zeros_like(W)
        e[i, j] = 1.0
        diff = (f(W + e) - f(W - e)) / 2
        assert abs(diff - float(G[i, j])) <= 1e-5 * float((dY.double().abs().t() @ x.abs())[i, j])


def test_weight_grad_strides_and_empty():
    t, n, k = 70, 130, 300
    q, s = mo.fp8_quantize(matrix(t, k, F32, 20))
    dY = matrix(t, n, BF16, 21)
    want = mo.fp8_weight_grad(dY, q, s, torch.empty((n, k), device="cuda"))
    bq = torch.full((t + 1, k + 13), 0x7F, dtype=torch.uint8, device="cuda")
    bs = torch.full((t + 1, 9), 255, dtype=torch.uint8, device="cuda")
    bq[:t, 3:3 + k] = F.codes(q)
    bs[:t, 2:5] = F.codes(s)
    by = torch.full((t + 1, n + 5), float("nan"), device="cuda", dtype=BF16)
    by[:t, 1:1 + n] = dY
    G = torch.full((n + 1, k + 3), 7.0, device="cuda")
    mo.fp8_weight_grad(by[:t, 1:1 + n], bq.view(F.FP8)[:t, 3:3 + k], bs.view(F.SCALE)[:t, 2:5], G[:n, 1:1 + k])
    assert torch.equal(G[:n, 1:1 + k], want)
    G[:n, 1:1 + k] = 7
    assert bool((G == 7).all())
    G = torch.ones((n, k), device="cuda")
    mo.fp8_weight_grad(dY[:0], q[:0], s[:0], G, accumulate=True)
    assert bool((G == 1).all())
    mo.fp8_weight_grad(dY[:0], q[:0], s[:0], G)
    assert bool((G == 0).all())
