"""The 8-bit products' plans on the CPU, from the library's own source compiled for the host
(host/fp8_plan.cpp): the cases of fp8_cases take the paths they are named for, and every path
that a wide grid of sizes reaches has a case."""
import itertools
import os
import shutil
import subprocess

import pytest

from fp8_cases import PRODUCTS, WGRADS

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="session")
def plans(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if cxx is None or not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("no host C++ compiler or no HIP headers")
    exe = str(tmp_path_factory.mktemp("plan") / "fp8_plan")
    subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "matrix_optimizers_amd", "csrc"),
                    os.path.join(HERE, "host", "fp8_plan.cpp"), "-o", exe, "-Wl,--unresolved-symbols=ignore-all"],
                   check=True, capture_output=True, text=True)

    def run(rows):
        text = "\n".join(" ".join(str(x) for x in r) for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(rows)
        got = []
        for line in out:
            p = {k: int(v) for k, v in (f.split("=") for f in line.split())}
            p["split"], p["many"] = int(p.pop("splits") > 1), int(p.pop("rounds") > 1)
            p["bytes"] = int(p["bytes"] > 0)
            if p.get("small"):
                p = {k: p[k] for k in ("small", "planes", "split", "bytes") if k in p and (k != "split" or "planes" in p)}
            got.append(p)
        return got
    return run


def product(m, n, k, f32, blk, off, inc):
    return "p", m, n, k, 0 if f32 else 1, blk, off, 0, 0, 0, inc


def wgrad(t, n, k, f32, off):
    return "w", t, n, k, 0 if f32 else 1, off, 0, 0, 0


def test_cases_take_the_paths_they_name(plans):
    got = plans([product(*c) for c, _ in PRODUCTS] + [wgrad(*c) for c, _ in WGRADS])
    for (c, want), p in zip(PRODUCTS + WGRADS, got):
        p = dict(p)
        needs = p.pop("bytes")
        assert {k: v for k, v in p.items() if v} == want, (c, p)
        # a workspace where something is copied, transposed or in parts, and only there
        parts = [want.get(k) for k in ("split", "copy_a", "copy_b", "scales_a", "scales_b")]
        assert needs == int(any(parts) or ("planes" in want and not want.get("tokens") and not want.get("small"))), c


def test_every_path_has_a_case(plans):
    tiles = ("small", "values", "tokens", "planes", "nb", "split", "many")
    copies = ("copy_a", "copy_b", "scales_a", "scales_b")

    def keys(rows):
        """The tiles' path, and what is copied."""
        for r, p in zip(rows, plans(rows)):
            for what in (tiles, copies):
                yield r, (r[0], what is tiles, *((k, p[k]) for k in what if p.get(k)))
    have = {k for _, k in keys([product(*c) for c, _ in PRODUCTS] + [wgrad(*c) for c, _ in WGRADS])}
    grid = [product(*c) for c in itertools.product((1, 70, 300, 700, 1030, 2100, 4133, 9000), (100, 260, 777, 1500, 2600, 5001),
                                                   (128, 500, 640, 1100, 2048, 4100, 8320, 16640), (0, 1), (1, 128), (0, 3), (0, 1))]
    grid += [wgrad(*c) for c in itertools.product((1, 64, 70, 300, 1030, 2100, 8000), (104, 264, 777, 1504, 2600, 5008),
                                                  (112, 272, 640, 1101, 2048, 4112), (0, 1), (0, 1))]
    missing = {k: r for r, k in keys(grid) if k not in have}
    assert not missing, missing
