"""Operands of 8-bit products and weight gradients large enough for the tiled kernels, in the layouts that
callers may have: every kind of tile, contiguous and in wider buffers.  test_fp8_layout_plans holds each to the
path that it names; test_fp8_tiles_gpu runs them.

A layout of a matrix in 8 bits: bytes by which its first row is off alignment, by how much rows are further
apart, the same two of its scales, and whether those lie by columns.  Of dY: elements off and further apart."""
from collections import namedtuple

Layout = namedtuple("Layout", "off pad soff spad cols", defaults=(0, 0, 0, 0, 0))
PLAIN = Layout()

Product = namedtuple("Product", "m n k f32 blk a b want")
Wgrad = namedtuple("Wgrad", "t n k f32 y x want")   # y: (off, pad) of dY


def blocks(n):
    return -(-n // 128)


def name(c):
    lay = lambda o: "+".join(map(str, o)) if any(o) else "0"
    if isinstance(c, Product):
        return f"{c.m}x{c.n}x{c.k}-{'f32' if c.f32 else 'bf16'}-{c.blk}-{lay(c.a)}-{lay(c.b)}"
    return f"{c.t}x{c.n}x{c.k}-{'f32' if c.f32 else 'bf16'}-{lay(c.y)}-{lay(c.x)}"


# in place and padded: rows stay whole 16 bytes, scales whole dwords
IN = Layout(16, 48, 4, 8), Layout(32, 4096, 8, 4)
# the rows in place, the scales not: by columns (with a stride of their own), or off alignment
BY_COLS, S_OFF = Layout(0, 16, 3, 5, 1), Layout(0, 0, 1, 3)
ODD = Layout(3, 5, 1, 3)

P = lambda m, n, k, f32, blk, a, b, **want: Product(m, n, k, f32, blk, a, b, want)
PRODUCTS = [
    # 8 bits, a weight's scales in blocks
    P(1030, 2600, 2048, 0, 128, PLAIN, PLAIN, nb=1),
    P(1030, 2600, 2048, 0, 128, IN[0], IN[1], nb=1),
    P(1030, 2600, 2048, 0, 128, BY_COLS, BY_COLS, nb=1, scales_a=1),
    P(1030, 2600, 2048, 0, 128, S_OFF, S_OFF, nb=1, scales_a=1),
    P(300, 5001, 8192, 0, 128, IN[1], BY_COLS, nb=1, split=1),
    P(9000, 260, 2048, 0, 128, IN[0], BY_COLS, nb=2),
    P(700, 1500, 16384, 0, 128, IN[0], IN[1], nb=2, split=1),
    P(4133, 5001, 640, 0, 128, IN[1], BY_COLS, nb=2, many=1, scales_a=1),
    P(9000, 777, 2048, 0, 128, IN[0], BY_COLS, nb=4),
    P(9000, 260, 16384, 0, 128, IN[0], IN[0], nb=4, split=1),
    P(4133, 5001, 8192, 0, 128, IN[1], BY_COLS, nb=4, split=1, many=1),
    # by rows
    P(1030, 2600, 2048, 0, 1, PLAIN, PLAIN, nb=1),
    P(1030, 2600, 2048, 0, 1, IN[0], IN[1], nb=1),
    P(1030, 2600, 2048, 0, 1, BY_COLS, BY_COLS, nb=1, scales_a=1, scales_b=1),
    P(300, 5001, 8192, 0, 1, IN[1], S_OFF, nb=1, split=1, scales_b=1),
    P(9000, 512, 2048, 0, 1, IN[0], BY_COLS, nb=2, scales_b=1),
    P(4133, 5001, 2048, 0, 1, IN[1], IN[0], nb=2, many=1),
    P(700, 1500, 16384, 0, 1, IN[0], IN[1], nb=2, split=1),
    P(9000, 777, 2048, 0, 1, IN[0], IN[1], nb=4),
    P(4133, 5001, 8192, 0, 1, IN[1], BY_COLS, nb=4, split=1, many=1, scales_b=1),
    # rows copied first
    P(1030, 2600, 1100, 0, 128, IN[0], IN[1], nb=1, copy_a=1, copy_b=1, scales_a=1),
    P(600, 5001, 2048, 0, 128, ODD, IN[0], nb=1, copy_a=1, scales_a=1),
    P(9000, 777, 1100, 0, 1, ODD, ODD, nb=4, copy_a=1, copy_b=1, scales_a=1, scales_b=1),
    # as bf16 numbers
    P(1030, 2600, 640, 1, 128, PLAIN, PLAIN, values=1, nb=1),
    P(1030, 2600, 640, 1, 128, IN[0], BY_COLS, values=1, nb=1),
    P(300, 1500, 16640, 1, 128, ODD, BY_COLS, values=1, nb=1, split=1),
    P(70, 5001, 128, 0, 1, ODD, BY_COLS, values=1, nb=1),
    P(9000, 260, 200, 1, 128, IN[0], BY_COLS, values=1, nb=2),
    P(700, 1500, 16640, 1, 1, BY_COLS, BY_COLS, values=1, nb=2, split=1),
    P(9000, 777, 200, 1, 1, ODD, BY_COLS, values=1, nb=4),
    P(4133, 5001, 128, 0, 128, ODD, BY_COLS, values=1, nb=4, many=1),
    P(4133, 777, 4100, 1, 128, ODD, ODD, values=1, nb=4, split=1),
]

W = lambda t, n, k, f32, y, x, **want: Wgrad(t, n, k, f32, y, x, want)
X_IN = Layout(16, 48, 1, 3), Layout(32, 4096, 0, 5)
Y_IN = (8, 24), (16, 4096)
WGRADS = [
    # read where they lie; the last stage has 6, 44, 52, 4 and 32 tokens, and one
    W(300, 1504, 2048, 0, (0, 0), PLAIN, tokens=1, planes=1, nb=1),
    W(300, 1504, 2048, 0, Y_IN[0], X_IN[0], tokens=1, planes=1, nb=1),
    W(2100, 264, 2048, 0, Y_IN[1], X_IN[1], tokens=1, planes=1, nb=1, split=1),
    W(70, 2600, 2048, 0, Y_IN[0], X_IN[1], tokens=1, planes=1, nb=2),
    W(4100, 1504, 640, 0, Y_IN[1], X_IN[0], tokens=1, planes=1, nb=2, split=1),
    W(70, 2600, 4112, 0, Y_IN[0], X_IN[0], tokens=1, planes=1, nb=4),
    W(96, 2600, 4112, 0, Y_IN[1], X_IN[1], tokens=1, planes=1, nb=4),
    W(65, 9000, 4112, 0, Y_IN[0], X_IN[0], tokens=1, planes=1, nb=4, many=1),
    W(1030, 9000, 2048, 0, Y_IN[0], X_IN[0], tokens=1, planes=1, nb=4, split=1, many=1),
    # transposed first
    W(1030, 264, 2048, 0, (1, 0), PLAIN, planes=1, nb=1),
    W(1030, 264, 2048, 0, (1, 7), BY_COLS, planes=1, nb=1),
    W(1030, 1504, 2048, 0, (0, 0), BY_COLS, planes=1, nb=1),
    W(2100, 777, 1101, 0, (0, 0), ODD, planes=1, nb=1, split=1),
    W(70, 777, 8016, 0, (0, 0), ODD, planes=1, nb=2),
    W(4100, 5008, 272, 0, (1, 3), BY_COLS, planes=1, nb=2, split=1),
    W(70, 9000, 1101, 0, (1, 3), ODD, planes=1, nb=4),
    W(4100, 9000, 2048, 0, (1, 3), BY_COLS, planes=1, nb=4, split=1, many=1),
    # an fp32 dY, in three planes
    W(300, 777, 4112, 1, (0, 0), PLAIN, planes=3, nb=1),
    W(300, 777, 4112, 1, (1, 3), BY_COLS, planes=3, nb=1),
    W(2100, 777, 1101, 1, (1, 3), ODD, planes=3, nb=1, split=1),
    W(300, 2600, 2048, 1, (1, 3), BY_COLS, planes=3, nb=2),
    W(2100, 777, 2048, 1, (0, 4), X_IN[0], planes=3, nb=2, split=1),
    W(70, 1504, 8016, 1, (1, 3), ODD, planes=3, nb=4),
    W(1030, 9000, 2048, 1, (1, 3), BY_COLS, planes=3, nb=4, split=1, many=1),
]


def strides(rows, cols, blk, lay):
    """offset ld offset_scales ld_scales inc_scales block_rows, as the binding passes them."""
    srows, scols = (rows if blk == 1 else blocks(rows)), blocks(cols)
    if lay.cols and scols > 1:
        return lay.off, cols + lay.pad, lay.soff, 1, srows + lay.spad, blk
    return lay.off, cols + lay.pad, lay.soff, (scols if not lay.cols else 1) + lay.spad, 0, blk
