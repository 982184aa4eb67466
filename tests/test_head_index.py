"""The output head's index functions as head_gemm.h has them: their text is taken from
the header and compiled for the host, so a change there is a change here.  And the
three-slot ring of its fp32 tile, with the waits read from the source."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = open(os.path.join(os.path.dirname(HERE), "matrix_optimizers_amd", "csrc", "head_gemm.h")).read()


def function(name):
    """Every definition of a function (templates and specialisations included), as text."""
    out = []
    for m in re.finditer(r"^(?:template <[^\n]*> )?(?:MO_DEV|inline) \w+ " + name + r"(?:<\d>)?\(", SOURCE, re.M):
        at, depth = SOURCE.index("{", m.start()), 0
        for i in range(at, len(SOURCE)):
            depth += {"{": 1, "}": -1}.get(SOURCE[i], 0)
            if depth == 0:
                out.append(SOURCE[m.start():i + 1])
                break
    assert out, name
    return "\n".join(out)


NAMES = ("seg_p", "seg_q", "hswz", "pswz", "qswz", "head_tile_of", "head_grid")
PROGRAM = r'''
#include <cstdint>
#include <cstdio>
#include <cstring>
#define MO_DEV inline
%s
int main(int argc, char** argv) {
    for (int r = 0; r < 256; ++r) std::printf("swz %%d %%d %%d %%d\n", r, hswz(r), pswz(r), qswz(r));
    for (int s = 0; s < 6; ++s) std::printf("seg 3 %%d %%d %%d\n", s, seg_p<3>(s), seg_q<3>(s));
    for (int s = 0; s < 2; ++s) std::printf("seg 2 %%d %%d %%d\n", s, seg_p<2>(s), seg_q<2>(s));
    std::printf("seg 1 0 %%d %%d\n", seg_p<1>(0), seg_q<1>(0));
    unsigned tm, tn;
    while (std::scanf("%%u %%u", &tm, &tn) == 2) {
        const uint32_t grid = head_grid(uint64_t(tm) * tn);
        std::printf("grid %%u %%u %%u\n", tm, tn, grid);
        for (uint32_t b = 0; b < grid; ++b) {
            uint32_t i = ~0u, j = ~0u;
            if (head_tile_of(b, tm, tn, i, j)) std::printf("tile %%u %%u %%u %%u %%u\n", tm, tn, b, i, j);
        }
    }
}
'''
SHAPES = [(1, 1), (1, 7), (3, 2), (5, 3), (8, 8), (126, 8), (501, 32), (9, 1), (1, 9), (125, 5), (4, 13), (7, 255), (501, 1)]


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("index")
    (d / "index.cpp").write_text(PROGRAM % "\n".join(function(n) for n in NAMES))
    subprocess.run([cxx, "-O1", "-std=c++17", str(d / "index.cpp"), "-o", str(d / "index")], check=True,
                   capture_output=True, text=True)
    out = subprocess.run([str(d / "index")], input="\n".join("%d %d" % s for s in SHAPES), capture_output=True, text=True,
                         check=True).stdout.splitlines()
    return [(f[0], *map(int, f[1:])) for f in (line.split() for line in out)]


def test_every_tile_runs_once(lines):
    for tm, tn in SHAPES:
        grid, = (x[3] for x in lines if x[:3] == ("grid", tm, tn))
        tiles = [x for x in lines if x[:3] == ("tile", tm, tn)]
        assert grid % 8 == 0 and grid - tm * tn < 8
        assert sorted(x[4:] for x in tiles) == [(i, j) for i in range(tm) for j in range(tn)]


def test_plane_pairs(lines):
    """Three planes each: the six largest products, the small ones first.  Two planes of P:
    what rounding left before the rounded value.  One: itself."""
    pairs = lambda planes: [x[3:] for x in sorted(lines) if x[:2] == ("seg", planes)]
    three = pairs(3)
    assert sorted(three) == [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (2, 0)]
    weight = [p + q for p, q in three]
    assert weight == sorted(weight, reverse=True)
    assert pairs(2) == [(1, 0), (0, 0)] and pairs(1) == [(0, 0)]


def bank_groups():
    """The sets of 16 lanes that the LDS serves together in a 16-byte read, as
    (row, K group): consecutive lanes, or four groups of four."""
    sets = [[(r, kg) for r in range(16)] for kg in range(4)]
    for kg in (0, 2):
        for a, b in ((kg, kg + 1), (kg + 1, kg)):
            sets.append([(r, a if r < 4 or r >= 12 else b) for r in range(16)])
    return sets


def test_swizzles_keep_the_banks_apart(lines):
    h, p, q = ({x[1]: x[2 + k] for x in lines if x[0] == "swz"} for k in range(3))
    for t, chunks in ((h, 8), (p, 8), (q, 4)):
        assert all(0 <= v < chunks for v in t.values())
    for lanes in bank_groups():
        for first in range(0, 256, 16):
            for c0 in (0, 4):        # 128-byte rows, chunk c0 + K group
                assert len({((first + r) * 128 + (((c0 + kg) ^ h[first + r]) << 4)) // 16 % 16 for r, kg in lanes}) == 16
            for half in (0, 1):      # fp32 rows, chunks 2 kg and 2 kg + 1
                assert len({((first + r) * 128 + (((2 * kg + half) ^ p[first + r]) << 4)) // 16 % 16 for r, kg in lanes}) == 16
            # 64-byte rows, chunk kg
            assert len({((first + r) * 64 + ((kg ^ q[first + r]) << 4)) // 16 % 16 for r, kg in lanes}) == 16
    # the fragment reads use the swizzle of row mod 16 for every row block
    assert all(t[r] == t[r % 16] for t in (h, p, q) for r in range(256))


# ---- the ring of head_tile32 -----------------------------------------------------------

def ring():
    """(slots, loads per stage, the prologue's waits, a stage's waits), from the source."""
    body = SOURCE[SOURCE.index("head_tile32(uint8_t* smem"):]
    slots = int(re.search(r"S32_SLOTS = (\d)", SOURCE).group(1))
    loads = 4 + int(re.search(r"constexpr int QI = (\d);", body).group(1))
    assert len(re.findall(r"raw_ptr_buffer_load_lds\(row, to", body)) == 1
    pro = re.search(r'if \(n > 2\) asm volatile\("s_waitcnt vmcnt\((\d+)\)".*?\n    else asm volatile\("s_waitcnt vmcnt\((\d+)\)"', body)
    stage = re.search(r'if \(s \+ 2 < n\) asm volatile\("s_waitcnt vmcnt\((\d+)\)".*?\n        else asm volatile\("s_waitcnt vmcnt\((\d+)\)"', body)
    # in a stage: the waits for loads and for its own reads, the barrier, then the refill and the reads
    order = [body.index(x) for x in ("if (s + 2 < n) asm volatile", "__builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)\n        __builtin_amdgcn_s_barrier();",
                                     "if (s + S < n) issue(s + S, slot);", "read(next, slot);")]
    assert order == sorted(order)
    return slots, loads, tuple(map(int, pro.groups())), tuple(map(int, stage.groups()))


def run_ring(n, slots, loads, pro, stage):
    """One wavefront's program order; every wavefront runs the same, so a barrier publishes
    what each of them has waited for, and ends every read before it."""
    issued = []          # stages, one entry per load
    landed = 0
    published, reading = set(), {}

    def issue(s):
        assert s % slots not in reading.values(), ("slot still being read", n, s)
        issued.extend([s] * loads)

    def wait(left):
        nonlocal landed
        landed = max(landed, len(issued) - left)

    def barrier():
        published.update(s for s in set(issued) if issued[:landed].count(s) == loads)
        reading.clear()

    def read(s):
        assert s in published, ("read before it has landed", n, s)
        assert max(x for x in issued if x % slots == s % slots) == s, ("slot refilled", n, s)
        reading[s] = s % slots

    for s in range(min(slots, n)):
        issue(s)
    wait(pro[0] if n > 2 else pro[1])
    barrier()
    read(0)
    for s in range(n):
        wait(stage[0] if s + 2 < n else stage[1])
        barrier()
        if s + slots < n:
            issue(s + slots)
        if s + 1 < n:
            read(s + 1)
    assert sorted(issued) == sorted(s for s in range(n) for _ in range(loads))


def test_ring_of_the_fp32_tile():
    for n in [*range(2, 41, 2), 64, 130]:
        run_ring(n, *ring())


@pytest.mark.parametrize("change", [dict(pro=(13, 7)), dict(pro=(12, 7)), dict(stage=(7, 0)), dict(stage=(6, 1)), dict(slots=2)])
def test_ring_model_catches_a_weaker_wait(change):
    slots, loads, pro, stage = ring()
    with pytest.raises(AssertionError):
        for n in range(2, 20, 2):
            run_ring(n, change.get("slots", slots), loads, change.get("pro", pro), change.get("stage", stage))
