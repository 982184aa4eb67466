"""Sizes of the 8-bit products and weight gradients, named by the path they take: what
test_fp8_plans holds to the plan and test_fp8_paths_gpu runs.

A product: rows of A, rows of B, K, whether the result is fp32, rows per scale of B, bytes by which
A's rows are off alignment, whether A's scales lie by columns; then its path: `small` (16 tb and 16 rb rows per
workgroup as tb rb) or tiles of 64 nb columns, as `values` or in 8 bits, K in parts (`split`), more than
one round of tiles (`many`), copies of A, of B and of their scales.
A weight gradient: tokens, rows, dim, fp32 dY, elements by which dY is off; its path: planes of dY, and blocks
of 64 x 64 (`small`) or tiles: read in place (`tokens`), nb, split, many."""

PRODUCTS = [
    ((70, 100, 500, 0, 128, 0, 0), dict(small=11)), ((70, 100, 500, 1, 128, 1, 0), dict(small=11)),
    ((3, 70, 33000, 0, 128, 0, 0), dict(small=11)), ((70, 100, 128, 0, 1, 0, 1), dict(small=12)),
    ((70, 100, 128, 1, 1, 0, 0), dict(small=12)), ((70, 260, 128, 0, 128, 0, 0), dict(small=22)),
    ((301, 600, 1408, 1, 128, 0, 0), dict(small=22)), ((70, 5001, 128, 0, 1, 0, 0), dict(small=44)),
    ((513, 2049, 2000, 1, 128, 5, 1), dict(small=22)), ((501, 2043, 2000, 1, 128, 0, 1), dict(small=44)), ((1030, 1500, 640, 0, 128, 0, 0), dict(small=44)),
    ((1030, 2600, 2048, 0, 1, 0, 0), dict(nb=1)), ((1030, 2600, 2048, 0, 128, 0, 0), dict(nb=1)),
    ((1030, 2600, 2048, 0, 1, 0, 1), dict(nb=1, scales_a=1)), ((1030, 2600, 128, 0, 128, 0, 0), dict(nb=1, scales_a=1)),
    ((1030, 2600, 128, 0, 1, 0, 0), dict(nb=1, scales_a=1, scales_b=1)), ((300, 5001, 2048, 0, 128, 3, 0), dict(nb=1, copy_a=1)),
    ((1030, 2600, 1100, 0, 128, 0, 0), dict(nb=1, copy_a=1, copy_b=1, scales_a=1)),
    ((1030, 2600, 1100, 0, 1, 0, 0), dict(nb=1, copy_a=1, copy_b=1, scales_a=1, scales_b=1)),
    ((300, 5001, 8320, 0, 128, 0, 0), dict(nb=1, split=1, scales_a=1)), ((700, 1500, 8320, 0, 1, 3, 0), dict(nb=1, split=1, copy_a=1, scales_a=1, scales_b=1)),
    ((4133, 777, 8320, 0, 128, 0, 0), dict(nb=1, split=1, many=1, scales_a=1)),
    ((4133, 777, 4100, 0, 1, 0, 0), dict(nb=1, split=1, many=1, copy_a=1, copy_b=1, scales_a=1, scales_b=1)),
    ((9000, 260, 2048, 0, 128, 0, 0), dict(nb=2)), ((9000, 260, 128, 0, 1, 0, 0), dict(nb=2, scales_a=1, scales_b=1)),
    ((4133, 777, 2048, 0, 128, 3, 1), dict(nb=2, copy_a=1, scales_a=1)), ((4133, 5001, 2048, 0, 1, 0, 0), dict(nb=2, many=1)),
    ((4133, 5001, 128, 0, 128, 0, 0), dict(nb=2, many=1, scales_a=1)), ((4133, 5001, 500, 0, 128, 0, 0), dict(nb=2, many=1, copy_a=1, copy_b=1)),
    ((700, 1500, 16640, 0, 128, 0, 0), dict(nb=2, split=1, scales_a=1)), ((9000, 777, 4100, 0, 128, 0, 0), dict(nb=2, split=1, many=1, copy_a=1, copy_b=1, scales_a=1)),
    ((9000, 777, 2048, 0, 1, 0, 0), dict(nb=4)), ((9000, 777, 1100, 0, 128, 0, 0), dict(nb=4, copy_a=1, copy_b=1, scales_a=1)),
    ((9000, 2600, 2048, 0, 128, 0, 0), dict(nb=4, many=1)), ((9000, 2600, 640, 0, 1, 3, 0), dict(nb=4, many=1, copy_a=1, scales_a=1, scales_b=1)),
    ((4133, 5001, 8320, 0, 128, 0, 0), dict(nb=4, split=1, many=1, scales_a=1)),
    ((4133, 5001, 8320, 0, 1, 3, 0), dict(nb=4, split=1, many=1, copy_a=1, scales_a=1, scales_b=1)),
    ((9000, 260, 16640, 0, 128, 0, 0), dict(nb=4, split=1, scales_a=1)), ((300, 1500, 16640, 1, 128, 3, 0), dict(values=1, nb=1, split=1)),
    ((70, 2600, 128, 1, 128, 3, 0), dict(values=1, nb=1)), ((70, 5001, 128, 0, 1, 3, 0), dict(values=1, nb=1)),
    ((9000, 260, 128, 1, 128, 0, 0), dict(values=1, nb=2)), ((9000, 260, 128, 0, 128, 3, 1), dict(values=1, nb=2)),
    ((700, 1500, 8320, 1, 128, 3, 1), dict(values=1, nb=2, split=1)), ((9000, 777, 4100, 1, 1, 0, 0), dict(values=1, nb=2, split=1, many=1)),
    ((9000, 777, 128, 1, 1, 0, 1), dict(values=1, nb=4)), ((4133, 5001, 128, 0, 128, 3, 0), dict(values=1, nb=4, many=1)),
    ((4133, 777, 4100, 1, 128, 0, 0), dict(values=1, nb=4, split=1)), ((4133, 5001, 2048, 1, 1, 0, 0), dict(values=1, nb=4, split=1, many=1)),
]

WGRADS = [
    ((1, 7, 3, 1, 1), dict(small=4, planes=3)),
    ((65, 129, 257, 0, 0), dict(small=4, planes=1)),
    ((300, 70, 1101, 1, 1), dict(small=4, planes=3)),
    ((700, 264, 272, 0, 1), dict(small=4, planes=1)),
    ((64, 5008, 2048, 1, 0), dict(small=4, planes=3)),
    ((1030, 1504, 112, 0, 1), dict(planes=1, nb=1)),
    ((1030, 64, 112, 0, 1), dict(planes=1, nb=1, split=1)),
    ((4100, 9000, 272, 0, 1), dict(planes=1, nb=1, split=1, many=1)),
    ((70, 777, 8016, 0, 0), dict(planes=1, nb=2)),
    ((1, 5008, 4112, 0, 1), dict(planes=1, nb=2, many=1)),
    ((8000, 5008, 112, 0, 1), dict(planes=1, nb=2, split=1)),
    ((2100, 9000, 2048, 0, 1), dict(planes=1, nb=2, split=1, many=1)),
    ((70, 9000, 1101, 0, 1), dict(planes=1, nb=4)),
    ((1, 9000, 8016, 0, 1), dict(planes=1, nb=4, many=1)),
    ((16000, 9000, 112, 0, 1), dict(planes=1, nb=4, split=1)),
    ((4100, 9000, 2048, 0, 1), dict(planes=1, nb=4, split=1, many=1)),
    ((300, 777, 4112, 1, 0), dict(planes=3, nb=1)),
    ((1030, 64, 112, 1, 0), dict(planes=3, nb=1, split=1)),
    ((300, 2600, 2048, 1, 1), dict(planes=3, nb=2)),
    ((70, 5008, 4112, 1, 1), dict(planes=3, nb=2, many=1)),
    ((8000, 2600, 112, 1, 0), dict(planes=3, nb=2, split=1)),
    ((1030, 5008, 2048, 1, 0), dict(planes=3, nb=2, split=1, many=1)),
    ((70, 1504, 8016, 1, 1), dict(planes=3, nb=4)),
    ((70, 9000, 8016, 1, 0), dict(planes=3, nb=4, many=1)),
    ((16000, 5008, 112, 1, 1), dict(planes=3, nb=4, split=1)),
    ((1030, 9000, 2048, 1, 0), dict(planes=3, nb=4, split=1, many=1)),
    ((300, 1504, 2048, 0, 0), dict(tokens=1, planes=1, nb=1)),
    ((1030, 64, 112, 0, 0), dict(tokens=1, planes=1, nb=1, split=1)),
    ((70, 2600, 2048, 0, 0), dict(tokens=1, planes=1, nb=2)),
    ((4100, 5008, 112, 0, 0), dict(tokens=1, planes=1, nb=2, split=1)),
    ((8000, 5008, 2048, 0, 0), dict(tokens=1, planes=1, nb=2, split=1, many=1)),
    ((1, 2600, 4112, 0, 0), dict(tokens=1, planes=1, nb=4)),
    ((1, 9000, 4112, 0, 0), dict(tokens=1, planes=1, nb=4, many=1)),
    ((8000, 9000, 112, 0, 0), dict(tokens=1, planes=1, nb=4, split=1)),
    ((1030, 9000, 2048, 0, 0), dict(tokens=1, planes=1, nb=4, split=1, many=1)),
    ((1, 64, 112, 0, 0), dict(small=4, planes=1)),
    ((1, 64, 112, 1, 0), dict(small=4, planes=3)),
]
