"""CPU models of the output head's GEMM (head_gemm.h): its K pipeline (the
schedule of the eight-wavefront core, checked by the same model at this core's
load counts), the cursor that walks the plane pairs of a split fp32 product, the
assignment of tiles to workgroups, and the rows its loads touch."""
import os
import re

import pytest

from test_gemm_pipeline import CSRC, check, wait_cases

HEADER = open(os.path.join(CSRC, "head_gemm.h")).read()


@pytest.mark.parametrize("LP", [8, 6])   # 2 (2 + QI): widths 256; 128 and 64
def test_pipeline_waits_are_exact_and_slots_safe(LP):
    cases, used = wait_cases("head_gemm.h"), set()
    for nk in range(8, 601, 2):
        used |= check(LP, nk)
    assert used <= cases


def test_short_products_fit_the_ring():
    """Two or four stages are loaded at once into the five slots; six never occur."""
    def k_extent(k):
        return 64 if k <= 64 else 128 if k <= 128 else max(256, (k + 63) // 64 * 64)
    for k in range(1, 5000):
        nk = k_extent(k) // 32
        assert nk % 2 == 0 and (nk in (2, 4) or nk >= 8), k
        assert k_extent(k) >= k
    # tokens padded to the tile width give a K extent too
    for n in range(1, 3000):
        nb = 1 if n <= 64 else 2 if n <= 128 else (2 if (n + 127) // 128 * 58 < (n + 255) // 256 * 100 else 4)
        n_pad = -(-n // (64 * nb)) * 64 * nb
        assert n_pad // 32 in (2, 4) or n_pad // 32 >= 8, n


def seg_tables():
    """The plane of P and Q in each of the six segments, read from the source."""
    body_p = re.search(r"int seg_p\(int s\) \{ return (.*?); \}", HEADER).group(1)
    body_q = re.search(r"int seg_q\(int s\) \{ return (.*?); \}", HEADER).group(1)
    def ev(expr, s):
        expr = expr.replace("PL == 1 ? 0 : ", "")
        m = re.match(r"s == (\d) \? 2 : \(s == (\d) \|\| s == (\d)\) \? 1 : 0", expr)
        a, b, c = map(int, m.groups())
        return 2 if s == a else 1 if s in (b, c) else 0
    return [(ev(body_p, s), ev(body_q, s)) for s in range(6)]


def test_plane_pairs_are_the_six_largest_smallest_first():
    pairs = seg_tables()
    assert sorted(pairs) == [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (2, 0)]
    weight = [a + b for a, b in pairs]
    assert weight == sorted(weight, reverse=True)


@pytest.mark.parametrize("nk1", [2, 4, 6, 8, 32])
def test_cursor_visits_every_stage_of_every_pair_in_order(nk1):
    """next_pair() after each pair of stages: stage s of the long loop is stage
    s mod nk1 of segment s / nk1."""
    ck, seg, off, seen = 0, 0, 0, []
    for _ in range(nk1 * 6 // 2):
        seen += [(seg, off), (seg, off + 1)]
        off += 2
        ck += 2
        if ck == nk1:
            ck, off, seg = 0, 0, seg + 1
    assert seen == [(s, k) for s in range(6) for k in range(nk1)]


def tile_of(b, tm, tn):
    nt, x, j = tm * tn, b & 7, b >> 3
    share, rem = nt >> 3, nt & 7
    if j >= share + (1 if x < rem else 0):
        return None
    t = x * share + min(x, rem) + j
    band = t // (4 * tn)
    r = t - band * 4 * tn
    h = min(4, tm - band * 4)
    return band * 4 + r % h, r // h


@pytest.mark.parametrize("tm,tn", [(1, 1), (1, 7), (3, 2), (5, 3), (8, 8), (501, 32), (9, 1), (125, 5), (4, 13)])
def test_every_tile_runs_once(tm, tn):
    grid = (tm * tn + 7) // 8 * 8
    tiles = [t for t in (tile_of(b, tm, tn) for b in range(grid)) if t]
    assert sorted(tiles) == [(i, j) for i in range(tm) for j in range(tn)]


@pytest.mark.parametrize("nb", [4, 2, 1])
def test_loads_fill_the_stage_and_stay_in_the_rows(nb):
    """The rows the eight waves' load instructions place in a stage, and the
    (clamped) rows they read for a matrix that ends inside the tile."""
    qi = 2 if nb == 4 else 1
    p_rows, q_rows = set(), set()
    for wave in range(8):
        qw = wave & 3 if nb == 1 else wave
        for lane in range(64):
            lrow = lane >> 2
            p_rows |= {wave * 32 + i * 16 + lrow for i in range(2)}
            q_rows |= {qw * 16 * qi + i * 16 + lrow for i in range(qi)}
    assert p_rows == set(range(256)) and q_rows == set(range(64 * nb))
    for have in (1, 17, 255, 256, 300):
        lim = min(have, 256) - 1
        assert max(min(r, lim) for r in p_rows) <= have - 1
