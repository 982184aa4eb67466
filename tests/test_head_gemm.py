"""CPU models of the output head's GEMM (head_gemm.h): the order in which a
wavefront issues its loads, reads fragments, waits and passes barriers; the
cursor that walks the plane pairs of a split fp32 product; the assignment of
tiles to workgroups; the rows and bytes its loads touch; its LDS swizzles; the
splitting of fp32 fragments."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "matrix_optimizers_amd", "csrc", "head_gemm.h")).read()
CPP = open(os.path.join(ROOT, "matrix_optimizers_amd", "csrc", "operators.cpp")).read()


def events(n, LS):
    """One wavefront's ('load', stage), ('read', stage), ('wait', left outstanding),
    ('barrier',) in program order, for n stages of LS loads each."""
    num, den = map(int, re.search(r"LH = \(LS \* (\d) \+ 7\) / (\d)", HEADER).groups())
    LH = (LS * num + 7) // den
    ev = [("load", 0)] * LS
    if n > 1:
        ev += [("load", 1)] * LS
    ev += [("wait", LS if n > 1 else 0), ("barrier",), ("read", 0)]     # first quarter's fragments

    def stage(s, ld0, nxt, ld3):
        # a quarter's reads and loads go out between its MFMAs: in any order
        out = [("read", s)]
        if ld0:
            out += [("load", s + 1)] * (LS - LH)
        out += [("read", s), ("read", s)]
        if nxt:
            out += [("wait", 0), ("barrier",), ("read", s + 1)]
        if ld3:
            out += [("load", s + 2)] * LH
        return out

    if n > 2:
        ev += stage(0, False, True, True)
        for s in range(1, n - 2):
            ev += stage(s, True, True, True)
        ev += stage(n - 2, True, True, False)
    elif n == 2:
        ev += stage(0, False, True, False)
    ev += stage(n - 1, False, False, False)
    return ev


def check(n, LS):
    ev = events(n, LS)
    loads = [e[1] for e in ev if e[0] == "load"]
    assert sorted(loads) == sorted(s for s in range(n) for _ in range(LS))
    issued, landed, published = [], 0, set()
    last_read = {}          # slot -> stage read since the last barrier
    free = {0: True, 1: True}   # slots no read is pending on
    for e in ev:
        if e[0] == "load":
            assert free[e[1] % 2], ("slot still being read", n, e)
            issued.append(e[1])
        elif e[0] == "wait":
            landed = max(landed, len(issued) - e[1])
        elif e[0] == "barrier":
            done = issued[:landed]
            published = {s for s in range(n) if done.count(s) == LS}
            free = {0: True, 1: True}
        else:
            assert e[1] in published, ("read before it is published", n, e)
            free[e[1] % 2] = False
    # the barrier that frees a slot comes after the last read of its stage
    for s in range(n - 2):
        first_load = max(i for i, e in enumerate(ev) if e == ("read", s))
        barrier = next(i for i, e in enumerate(ev) if i > first_load and e == ("barrier",))
        refill = next(i for i, e in enumerate(ev) if e == ("load", s + 2))
        assert barrier < refill, (n, s)


@pytest.mark.parametrize("LS", [8, 6, 5])   # 4 + NB load instructions per stage
def test_pipeline(LS):
    for n in list(range(1, 40)) + [64, 129]:
        check(n, LS)


def test_model_catches_an_early_refill(monkeypatch):
    orig = events

    def bad(n, LS):
        ev = orig(n, LS)
        i = next(i for i, e in enumerate(ev) if e == ("load", 2))
        return ev[:5] + [ev[i]] + ev[5:i] + ev[i + 1:]
    import sys
    monkeypatch.setattr(sys.modules[__name__], "events", bad)
    with pytest.raises(AssertionError):
        check(8, 8)


def test_waits_cover_the_load_counts():
    """The prologue leaves exactly the second stage's LS = 4 + NB loads outstanding."""
    assert re.search(r"LS = 4 \+ NB;", HEADER)
    for ls in (8, 6):
        assert f"if constexpr (LS == {ls}) asm volatile(\"s_waitcnt vmcnt({ls})\"" in HEADER
    assert "else asm volatile(\"s_waitcnt vmcnt(5)\"" in HEADER


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


@pytest.mark.parametrize("nk1", [1, 2, 3, 8, 33])
def test_cursor_visits_every_stage_of_every_pair_in_order(nk1):
    """next_stage() after each stage: stage s of the long loop is stage s mod nk1 of
    segment s / nk1."""
    ck, seg, off, seen = 0, 0, 0, []
    for _ in range(nk1 * 6):
        seen.append((seg, off))
        off += 1
        ck += 1
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


def swz(row):
    return (row >> 1) & 7


@pytest.mark.parametrize("nb", [4, 2, 1])
def test_loads_fill_the_stage_and_stay_in_the_rows(nb):
    """The bytes the eight waves' load instructions place in a stage, which chunk of
    which row each is, and the (clamped) rows they read for a matrix that ends
    inside the tile."""
    filled = {}
    for wave in range(8):
        for i in range(4 + nb):
            first = wave * 32 + i * 8 if i < 4 else wave * 8 * nb + (i - 4) * 8
            base = first * 128 + (0 if i < 4 else 256 * 128)
            for lane in range(64):
                r = first + (lane >> 3)
                at = base + lane * 16
                assert at not in filled
                filled[at] = (i >= 4, r, (lane & 7) ^ swz(r))
    assert sorted(filled) == list(range(0, (256 + 64 * nb) * 128, 16))
    # where the fragment reads look for chunk c of row r
    for q, rows in ((False, 256), (True, 64 * nb)):
        for r in range(rows):
            for c in range(8):
                assert filled[(256 * 128 if q else 0) + r * 128 + ((c ^ swz(r)) << 4)] == (q, r, c)
    for have in (1, 17, 255, 256, 300):
        lim = min(have, 256) - 1
        assert max(min(r, lim) for r in range(256)) <= have - 1


def test_fragment_reads_hit_distinct_banks():
    """64 lanes read 16 rows x chunks c .. c + 3 (c = 0 or 4): the sixteen lanes served
    together, consecutive or four groups of four, lie in distinct 16-byte groups
    of the 256-byte bank line."""
    for c0 in (0, 4):
        addr = [(l & 15) * 128 + (((c0 + (l >> 4)) ^ swz(l & 15)) << 4) for l in range(64)]
        groups = [range(16 * g, 16 * g + 16) for g in range(4)]
        for h in (0, 32):
            groups.append([h + x for x in list(range(0, 4)) + list(range(12, 16)) + list(range(20, 28))])
            groups.append([h + x for x in list(range(4, 12)) + list(range(16, 20)) + list(range(28, 32))])
        for g in groups:
            assert len({addr[l] // 16 % 16 for l in g}) == 16, (c0, list(g))


def test_copy_strides_cover_their_extents():
    """copy_stride(k) holds k elements and is never a multiple of 4 KB."""
    assert "k * 2 % 4096 == 0 ? k + 64 : k" in CPP
    for k in range(64, 70000, 64):
        ld = k + 64 if k * 2 % 4096 == 0 else k
        assert ld >= k and ld * 2 % 4096 != 0 and ld * 2 % 128 == 0


def test_fp32_fragments_split_exactly():
    """The integer form of the three planes: nearest with ties away from zero, finite
    high parts, and nothing left over."""
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.integers(-30, 30, 20000),
                        [0.0, -0.0, 1.0, 3.4028235e38, -3.4028235e38, 3.3895314e38, 1 + 2.0 ** -8, 1 + 2.0 ** -9]])
    x = x.astype(np.float32)
    top = np.float32(3.3895313892515355e38)

    def near(v):
        return ((v.view(np.uint32) + np.uint32(0x8000)) & np.uint32(0xFFFF0000)).view(np.float32)

    h = near(np.clip(x, -top, top))
    r = x - h
    m = near(r)
    low = r - m
    assert np.isfinite(h).all()
    # the last of 24 bits is 2^-23 of the first, and bf16 ends at 2^-133
    assert ((low.view(np.uint32) & 0xFFFF) == 0)[np.abs(x) >= 2.0 ** -109].all()
    assert (h.astype(np.float64) + m + low == x).all()
    assert (np.abs(m) <= 2.0 ** -7 * np.abs(x)).all() and (np.abs(low) <= 2.0 ** -15 * np.abs(x)).all()


def test_in_place_fragments_reach_every_bank_once():
    """The swizzles of the fp32 tiles: each set of 16 lanes served together falls on
    16 different 16-byte bank groups, for every chunk it reads."""
    def pswz(r):
        x = r >> 1
        return ((x << 1) & 6) | ((x >> 2) & 1)

    def qswz(r):
        g = (r >> 2) & 3
        return ((g << 1) & 2) ^ ((g >> 1) * 3)

    assert sorted(pswz(2 * i) for i in range(8)) == list(range(8))
    assert sorted(qswz(4 * i) for i in range(4)) == list(range(4))
    sets = [[(r, kg) for r in range(16)] for kg in range(4)]
    for kg in (0, 2):
        for a, b in ((kg, kg + 1), (kg + 1, kg)):
            sets.append([(r, a if r < 4 or r >= 12 else b) for r in range(16)])
    for lanes in sets:
        for half in (0, 1):
            assert len({(r * 128 + (((2 * kg + half) ^ pswz(r)) << 4)) % 256 // 16 for r, kg in lanes}) == 16
        assert len({(r * 64 + ((kg ^ qswz(r)) << 4)) % 256 // 16 for r, kg in lanes}) == 16
    # K along the rows: 64 lanes on 64 banks
    for wave in range(8):
        for a in (0, 1):
            for e in range(8):
                at = [(kg * 8 + e) * 1024 + ((((wave * 32 + a * 16 + r) >> 2) ^ (kg << 2)) << 4) + (r & 3) * 4
                      for kg in range(4) for r in range(16)]
                assert len({x % 256 // 4 for x in at}) == 64
                # and each holds its own element: chunk c of row k at c ^ 4 (k / 8 mod 4)
                for i, x in enumerate(at):
                    k, chunk = x // 1024, x % 1024 // 16
                    assert ((chunk ^ (((k >> 3) & 3) << 2)) * 4 + x % 16 // 4) == wave * 32 + a * 16 + i % 16
