"""What include/mo.h says of the 8-bit products' and weight gradients' paths, on the CPU."""
from fp8_layouts import Layout, PLAIN, strides
from test_fp8_layout_plans import plan  # noqa: F401  (a fixture)

ODD = Layout(3, 5, 1, 3)


def test_small_bf16_products_are_in_8_bits_whatever_their_alignment(plan):  # noqa: F811
    for m, n, k in ((1, 5, 127), (8, 4096, 4096), (70, 300, 500), (200, 1000, 1000)):
        for a, b in ((PLAIN, PLAIN), (ODD, ODD), (ODD, PLAIN)):
            for blk in (1, 128):
                assert plan(["p", m, n, k, 1, *strides(m, k, 1, a), *strides(n, k, blk, b)]).get("small"), (m, n, k, a, b)
