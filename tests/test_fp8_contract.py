"""What include/mo.h says of the 8-bit products' and weight gradients' strides and paths, on the CPU."""
import pytest

from fp8_layouts import Layout, PLAIN, strides
from test_fp8_abi import A, OK, UNSUPPORTED, act, mm, mm_bytes, wei, wg, wg_bytes
from test_fp8_layout_plans import plan  # noqa: F401  (a fixture)

ODD = Layout(3, 5, 1, 3)


def x(**kw):
    return wei(500, block_rows=1, **kw)


@pytest.mark.parametrize("ld", [(1 << 23) - 1, 1 << 23, (1 << 24) + 8, 1 << 25, 1 << 26])
def test_a_weight_gradient_takes_strides_up_to_2_26(ld):
    for kw in (dict(x=x(ld_q=ld)), dict(x=x(ld_scales=ld)), dict(x=x(ld_scales=1, inc_scales=ld)), dict(ldy=ld), dict(ldy=ld, yt=0)):
        assert wg_bytes(**kw)[0] == OK
    for kw in (dict(ldg=ld), dict(ldg=ld, gt=1)):   # accepted up to the check behind the strides'
        assert wg(have=0, x=wei(16384, block_rows=1), **kw) not in (OK, UNSUPPORTED)


@pytest.mark.parametrize("kw", [dict(x=x(ld_q=(1 << 26) + 1)), dict(x=x(ld_scales=(1 << 26) + 1)),
                                dict(x=x(ld_scales=1, inc_scales=(1 << 26) + 1)), dict(ldy=(1 << 26) + 1)])
def test_and_no_longer_ones(kw):
    assert wg_bytes(**kw)[0] == UNSUPPORTED and wg(**kw) == UNSUPPORTED


def test_a_product_takes_strides_below_2_23():
    top = (1 << 23) - 1
    assert mm_bytes(act(ld_q=top), wei(ld_scales=top), 512) >= 0
    for a, b in ((act(ld_q=top + 1), wei()), (act(ld_scales=top + 1), wei()), (act(), wei(ld_q=top + 1)), (act(), wei(ld_scales=top + 1))):
        assert mm(a, b, Y=A[4]) == UNSUPPORTED
    # columns of scales, and Y's rows, as elsewhere
    assert mm_bytes(act(ld_scales=1, inc_scales=1 << 26), wei(ld_scales=1, inc_scales=1 << 26), 512) >= 0
    assert mm(long_a := act(1500), wei(1000), 16384, ldy=1 << 26, have=0) not in (OK, UNSUPPORTED) and long_a.rows == 1500


def test_small_bf16_products_are_in_8_bits_whatever_their_alignment(plan):  # noqa: F811
    for m, n, k in ((1, 5, 127), (8, 4096, 4096), (70, 300, 500), (200, 1000, 1000)):
        for a, b in ((PLAIN, PLAIN), (ODD, ODD), (ODD, PLAIN)):
            for blk in (1, 128):
                assert plan(["p", m, n, k, 1, *strides(m, k, 1, a), *strides(n, k, blk, b)]).get("small"), (m, n, k, a, b)


def test_the_longest_strides_take_the_tiles_they_are_tested_for(plan):  # noqa: F811
    """Those of test_fp8_strides_gpu."""
    def lay(k, ld, lds):
        return Layout(0, ld - k, 0, lds - -(-k // 128), 0)
    top = (1 << 23) - 16, (1 << 23) - 4
    for m, n, k, t, blk, ld, want in ((1030, 2600, 2048, 1, 128, top, dict(nb=1)), (1030, 2600, 2048, 1, 1, top, dict(nb=1)),
                                      (1030, 2600, 640, 0, 128, ((1 << 23) - 1,) * 2, dict(values=1, nb=1))):
        assert plan(["p", m, n, k, t, *strides(m, k, 1, lay(k, *ld)), *strides(n, k, blk, lay(k, *ld))]) == want
    inside, most = ((1 << 24) - 8, (1 << 25) - 16, (1 << 25) - 1), ((1 << 26) - 1, 1 << 26, 1 << 26)
    for t, n, k, y, (ldy, ld, lds), want in ((300, 1504, 2048, 1, inside, dict(tokens=1, planes=1, nb=1)),
                                             (70, 2600, 2048, 1, inside, dict(tokens=1, planes=1, nb=2)),
                                             (70, 2600, 4112, 1, inside, dict(tokens=1, planes=1, nb=4)),
                                             (70, 9000, 1101, 1, most, dict(planes=1, nb=4)),
                                             (70, 1504, 8016, 0, most, dict(planes=3, nb=4))):
        assert plan(["w", t, n, k, y, 0, ldy, *strides(t, k, 1, lay(k, ld, lds))]) == want
