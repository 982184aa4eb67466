"""Plain 64-bit forms of the RMS norm and of the 8-bit operators, written from their
formulas, with element-wise bounds (the conventions of operators_ref)."""
import torch

from operators_ref import U, norm_depth, ut

BLOCK = 128
FP8, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


def blocks(n):
    return -(-n // BLOCK)


def codes(t):
    """The bytes of a float8 tensor."""
    return t.view(torch.uint8)


def bytes_of(amax):
    """The least b >= 0 with amax <= 448 2^(b - 127), by trying around the logarithm."""
    a = amax.double()
    b = torch.floor(torch.log2(a.clamp(min=1e-300) / 448)) + 127
    for _ in range(3):
        b = torch.where(a > 448 * torch.exp2(b - 127), b + 1, b)
    for _ in range(3):
        b = torch.where((a <= 448 * torch.exp2(b - 128)), b - 1, b)
    return torch.where(a > 0, b, torch.zeros_like(b)).clamp(min=0)


def row_amax(x):
    """Largest finite magnitude of each block of a row (rows, blocks)."""
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).double().abs()
    return torch.stack([x[:, c:c + BLOCK].amax(1) for c in range(0, x.shape[1], BLOCK)], 1)


def square_amax(x):
    a = row_amax(x)
    return torch.stack([a[r:r + BLOCK].amax(0) for r in range(0, x.shape[0], BLOCK)], 0)


def spread(b, rows, cols, r=1):
    """Per element from per block of r rows."""
    i = torch.arange(rows, device=b.device) // r
    j = torch.arange(cols, device=b.device) // BLOCK
    return b[i][:, j]


def e4m3(v):
    """v (float64) on e4m3's numbers, ties to even; not finite: NaN."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.where(torch.isfinite(v), torch.round(v / step) * step, torch.full_like(v, float("nan")))


def quantize(x, r=1):
    """(q, bytes) of x as float64."""
    b = bytes_of(row_amax(x) if r == 1 else square_amax(x))
    return e4m3(x.double() * torch.exp2(127 - spread(b, *x.shape, r))), b


def value(q, s, r=1):
    return q.double() * spread(s.double(), q.shape[0], q.shape[1], r)


# ---- RMS norm ------------------------------------------------------------------------

def rms(h, w, eps):
    x = h.double()
    r = (x.square().mean(1) + eps) ** -0.5
    y = x * r[:, None]
    return (y if w is None else y * w.double()), r


def rms_r_bound(cols):
    """Of r, relative: the sum's D additions and squares, the quotient, eps and the square
    root, half of that; then the root and the quotient."""
    return (0.5 * (norm_depth(cols) + 4) + 3) * U


def rms_grad(dY, h, r, w, dH):
    x, g, r = h.double(), dY.double(), r.double()[:, None]
    gw = g if w is None else g * w.double()
    xh = x * r
    n = x.shape[1]
    m = (gw * xh).sum(1, keepdim=True) / n
    dx = r * (gw - xh * m)
    # the sum has D additions and three products, each of m's own terms; then five roundings
    d = norm_depth(n) + 5
    b = r * (4 * U * gw.abs() + xh.abs() * ((d + 4) * U * (gw * xh).abs().sum(1, keepdim=True) / n))
    if dH is not None:
        dx = dx + dH.double()
        b = b + U * dH.double().abs()
    b = b + ut(h.dtype) * dx.abs()
    p = g * xh
    return (dx, p.sum(0)), (b, (x.shape[0] + 4) * U * p.abs().sum(0))


# ---- products ------------------------------------------------------------------------

def matmul(A, sa, B, sb, ra, rb, dtype):
    """Y and its bound.  fp32: K additions of 2 u each on the matrix cores and the splits'.  bf16: each
    instruction's 128 products are kept to 2^-16 of the largest (an eighth of it, over 128, is
    2^-9 of a block's largest product, itself at most the product of both rows' largest)."""
    a, b = value(A, sa, ra), value(B, sb, rb)
    Y = a @ b.t()
    M = a.abs() @ b.abs().t()
    K = A.shape[1]
    if dtype == torch.float32:
        return Y, (K + 64) * 2 * U * M
    pa = torch.stack([a[:, c:c + BLOCK].abs().amax(1) for c in range(0, K, BLOCK)], 1)
    pb = torch.stack([b[:, c:c + BLOCK].abs().amax(1) for c in range(0, K, BLOCK)], 1)
    return Y, 2.0 ** -9 * (pa @ pb.t()) + (blocks(K) + 64) * 2 * U * M + ut(dtype) * Y.abs()


def wgrad(dY, q, s, dtype, G=None):
    x, g = value(q, s), dY.double()
    W = g.t() @ x
    planes = 3 if dY.dtype == torch.float32 else 1
    b = (planes * dY.shape[0] + 64) * 2 * U * (g.abs().t() @ x.abs()) * (1 + 2.0 ** -6)
    if G is not None:
        W = W + G.double()
        b = b + U * W.abs()
    return W, b + ut(dtype) * W.abs()
