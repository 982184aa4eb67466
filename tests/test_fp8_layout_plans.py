"""The cases of fp8_layouts take the tiles that they are named for (the library's plan, compiled for
the host), so that a change of the choice between the kernels shows."""
import os
import shutil
import subprocess

import pytest

from fp8_layouts import PRODUCTS, WGRADS, name, strides

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if cxx is None or not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("no host C++ compiler or no HIP headers")
    exe = str(tmp_path_factory.mktemp("plan") / "fp8_layout_plan")
    subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "matrix_optimizers_amd", "csrc"),
                    os.path.join(HERE, "host", "fp8_layout_plan.cpp"), "-o", exe, "-Wl,--unresolved-symbols=ignore-all"],
                   check=True, capture_output=True, text=True)

    def run(row):
        out = subprocess.run([exe], input=" ".join(map(str, row)), capture_output=True, text=True, check=True).stdout
        return {k: int(v) for k, v in (f.split("=") for f in out.split()) if int(v)}
    return run


@pytest.mark.parametrize("c", PRODUCTS, ids=name)
def test_product(plan, c):
    assert plan(["p", c.m, c.n, c.k, 0 if c.f32 else 1, *strides(c.m, c.k, 1, c.a), *strides(c.n, c.k, c.blk, c.b)]) == c.want


@pytest.mark.parametrize("c", WGRADS, ids=name)
def test_weight_grad(plan, c):
    es = 4 if c.f32 else 2
    assert plan(["w", c.t, c.n, c.k, 0 if c.f32 else 1, c.y[0] * es, c.n + c.y[1], *strides(c.t, c.k, 1, c.x)]) == c.want


def test_every_kind_of_tile_is_there():
    """Each kind, width, and K whole or in parts; each in a buffer wider than the matrix."""
    have = {("values" if c.want.get("values") else "square" if c.blk == 128 else "rows", c.want["nb"], c.want.get("split", 0))
            for c in PRODUCTS if any(c.a) and any(c.b)}
    for kind in ("square", "rows", "values"):
        for nb in (1, 2, 4):
            assert {(kind, nb, 0), (kind, nb, 1)} <= have, (kind, nb)
    have = {("tokens" if c.want.get("tokens") else c.want["planes"], c.want["nb"], c.want.get("split", 0))
            for c in WGRADS if any(c.y) or any(c.x)}
    for kind in ("tokens", 1, 3):
        for nb in (1, 2, 4):
            assert {(kind, nb, 0), (kind, nb, 1)} <= have, (kind, nb)
    last = {c.t % 64 for c in WGRADS if c.want.get("tokens")}
    assert min(last) == 1 and any(1 < x <= 32 for x in last) and any(x > 32 for x in last)
