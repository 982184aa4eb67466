"""The output head's plans on the CPU, from the library's own source compiled for the
host (host/head_plan.cpp): the cases of head_cases.py take the paths they are named
for."""
import os
import shutil
import subprocess

import pytest

from head_cases import BF16, CASES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="session")
def planner(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if cxx is None or not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("no host C++ compiler or no HIP headers")
    exe = str(tmp_path_factory.mktemp("plan") / "head_plan")
    subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "matrix_optimizers_amd", "csrc"),
                    os.path.join(HERE, "host", "head_plan.cpp"), "-o", exe, "-Wl,--unresolved-symbols=ignore-all"],
                   check=True, capture_output=True, text=True)

    def plans(rows):
        """One dict per (tokens, vocab, dim, dtype code, backward, k, ld_h, ld_w, h offset, w offset)."""
        text = "\n".join(" ".join(str(x) for x in r) for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(rows)
        got = [{k: int(v) for k, v in (f.split("=") for f in line.split())} for line in out]
        for p in got:
            if p["status"] == 0:
                p["split"], p["many"] = int(p["z_splits"] > 1), int(p["pieces"] > 1)
        return got
    return plans


@pytest.mark.parametrize("name", CASES)
def test_cases_take_the_paths_they_name(planner, name):
    dtype, n, vocab, dim, *want = CASES[name]
    for back, w in enumerate(want):
        got = planner([(n, vocab, dim, 1 if dtype == BF16 else 0, back, 1, 0, 0, 0, 0)])[0]
        assert {k: got[k] for k in w} == w, (name, "backward" if back else "forward", got)


def test_every_path_has_a_case(planner):
    """Tile widths, delta's planes, split K, several pieces: each combination that the sizes
    of a wide grid reach is that of some case, in the backward plan."""
    key = lambda p: (p["planes"], p["dt_planes"], p["f32w"], p["nb"], p["split"], p["many"])
    have = set()
    for dtype, n, vocab, dim, _, _ in CASES.values():
        have.add(key(planner([(n, vocab, dim, 1 if dtype == BF16 else 0, 1, 1, 0, 0, 0, 0)])[0]))
    rows = [(n, v, d, t, 1, 1, 0, 0, 0, 0) for n in (1, 40, 65, 128, 129, 257, 513, 700, 1345, 2049, 8192)
            for v in (300, 1984, 10001, 32001, 60001, 100003, 131072) for d in (64, 100, 233, 1024, 2500, 4096, 7354)
            for t in (0, 1)]
    missing = {}
    for r, p in zip(rows, planner(rows)):
        if key(p) not in have:
            missing.setdefault(key(p), r)
    assert not missing, missing


def test_two_planes_of_delta_go_with_narrow_tiles_and_whole_sums(planner):
    """The kernels for delta in two planes are built for tiles of 64 and 128 tokens and a
    dW whose K is not split."""
    rows = [(n, v, d, 1, 1, 1, 0, 0, 0, 0) for n in (1, 2, 63, 64, 65, 100, 127, 128, 129)
            for v in (1, 300, 5000, 32001, 131072, 1 << 20, 1 << 24) for d in (1, 64, 128, 129, 1000, 4096, 65536)]
    for r, p in zip(rows, planner(rows)):
        assert p["dt_planes"] == (2 if r[0] <= 128 else 1)
        if p["dt_planes"] == 2:
            assert p["nb"] <= 2 and p["dw_splits"] == 1, (r, p)


def test_which_operands_are_read_as_they_lie(planner):
    """bf16: rows of whole 128 bytes at 16-byte addresses less than 8 MB apart; fp32 with at
    most 512 tokens: W's rows of whole 16 bytes, likewise.  Everything else is copied."""
    def packs(dtype, n=40, dim=128, ldh=0, ldw=0, oh=0, ow=0):
        p = planner([(n, 300, dim, dtype, 0, 1, ldh, ldw, oh, ow)])[0]
        return p["pack_h"], p["pack_w"]
    assert packs(1) == (0, 0) and packs(1, ldh=136, ldw=192, oh=8, ow=16) == (0, 0)
    assert packs(1, ldh=132) == (1, 0) and packs(1, ldw=129) == (0, 1)
    assert packs(1, oh=4) == (1, 0) and packs(1, ow=1) == (0, 1)
    assert packs(1, dim=100) == packs(1, dim=192 + 8) == (1, 1)
    assert packs(1, ldw=(1 << 22) - 8) == (0, 0) and packs(1, ldw=1 << 22) == (0, 1)
    assert packs(0) == packs(0, dim=100) == packs(0, ldw=132, ow=4) == (1, 0)
    assert packs(0, dim=99) == packs(0, ldw=130) == packs(0, ow=2) == packs(0, ldw=1 << 21) == (1, 1)
    assert packs(0, n=512) == (1, 0) and packs(0, n=513) == (1, 1)


def test_pieces_and_copies_hold_what_they_are_for(planner):
    """Pieces are whole tiles that cover the vocabulary; splits of K cover it; copies'
    rows are whole stages."""
    rows = [(n, v, d, t, b, 1, 0, 0, 0, 0) for n in (1, 64, 65, 128, 129, 512, 513, 8192, 1 << 20)
            for v in (1, 256, 257, 32001, 131072, 1 << 22) for d in (1, 63, 64, 65, 1000, 4096, 65536)
            for t in (0, 1) for b in (0, 1)]
    for (n, v, d, *_), p in zip(rows, planner(rows)):
        assert p["piece"] % 256 == 0 and (p["pieces"] - 1) * p["piece"] < v <= p["pieces"] * p["piece"]
        assert p["n_pad"] % (64 * p["nb"]) == 0 and 0 <= p["n_pad"] - n < 64 * p["nb"]
        assert p["kd"] % 64 == 0 and 0 <= p["kd"] - d < 64
        assert p["z_splits"] * p["z_stages"] >= p["kd"] // 64 > (p["z_splits"] - 1) * p["z_stages"]
