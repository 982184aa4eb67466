"""Every launch of the operators stays inside one launch's limits (fewer than 2^32
threads along an axis, 65535 workgroups along y, 1024 threads in a workgroup, none
empty) at the largest sizes the entry points accept, alone and together.  The built
library runs against a stand-in for the runtime's launches (host/fake_hip.cpp), loaded
before it, that records them instead of making them; the addresses are never used."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(ROOT, "matrix_optimizers_amd", "libmo.so")

CHILD = r'''
import ctypes, itertools, sys
fake = ctypes.CDLL(sys.argv[2], mode=ctypes.RTLD_GLOBAL)   # found before the library's own dependencies
lib = ctypes.CDLL(sys.argv[1])
P, I, N, F, Z = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t

class Head(ctypes.Structure):
    _fields_ = [(n, P) for n in ("H", "W")] + [(n, I) for n in ("tokens", "vocab", "dim", "ld_h", "ld_w")] + [("dtype", N)]

class Topk(ctypes.Structure):
    _fields_ = [("ids", P), ("logits", P), ("ld_ids", I), ("ld_logits", I), ("k", N), ("dtype", N), ("temperature", F)]

HUGE = 1 << 59
A = [P(k << 59) for k in range(1, 31)]       # addresses no range of these sizes joins
def take(what, st):
    out = (ctypes.c_uint64 * 6)()
    fake.fake_hip_take(out)
    print(what, st, *out, flush=True)

def edges(*axes):
    return itertools.product(*axes)

for n, v, d, t in edges((1, 1 << 30), (1, 1 << 27), (1, 1 << 20), (0, 1)):
    st = lib.embedding_forward(A[0], I(n), A[1], I(0), I(v), I(d), N(t), F(1), A[2], I(0), None)
    take(f"embedding_forward {n}x{v}x{d}:{t}", st)
    st = lib.embedding_backward(A[0], I(n), A[1], I(0), N(t), A[2], I(0), N(t), I(v), I(d), F(1), N(0), A[3], Z(HUGE), None)
    take(f"embedding_backward {n}x{v}x{d}:{t}", st)
for r, c, t in edges((1, 1 << 32), (1, 512, 16384, 1 << 24), (0, 1)):
    st = lib.layer_norm_forward(A[0], I(0), A[1], A[2], A[3], I(0), A[4], A[5], I(r), I(c), N(t), F(1e-5), None)
    take(f"layer_norm_forward {r}x{c}:{t}", st)
    st = lib.layer_norm_backward(A[0], I(0), A[1], I(0), A[2], A[3], A[4], A[5], I(0), A[6], A[7], I(r), I(c), N(t), A[8], Z(HUGE), None)
    take(f"layer_norm_backward {r}x{c}:{t}", st)
T, V, D = 1 << 20, 1 << 26, 1 << 16
sizes = [(1, 1, 1), (T, 1, 1), (1, V, 1), (1, 1, D), (T, 1, D), (T, 1 << 16, D), (1, V, D), (T, 300, 16384), (T, 1 << 22, 64),
         (128, V, 64), (4096, V, 4096), (513, V, 1000)]
for (n, v, d), t in edges(sizes, (0, 1)):
    h = Head(A[0], A[1], n, v, d, 0, 0, t)
    st = lib.softmax_xent_forward(ctypes.byref(h), A[2], A[3], A[4], A[5], Z(HUGE), None)
    take(f"softmax_xent_forward {n}x{v}x{d}:{t}", st)
    st = lib.softmax_xent_backward(ctypes.byref(h), A[2], A[3], A[4], A[5], A[6], I(0), A[7], I(0), A[8], Z(HUGE), None)
    take(f"softmax_xent_backward {n}x{v}x{d}:{t}", st)
    k = Topk(A[2], A[3], 0, 0, 1024, t, 1.0)
    st = lib.topk_distill_forward(ctypes.byref(h), ctypes.byref(k), A[4], A[5], A[6], A[7], Z(HUGE), None)
    take(f"topk_distill_forward {n}x{v}x{d}:{t}", st)
    st = lib.topk_distill_backward(ctypes.byref(h), ctypes.byref(k), A[4], A[5], A[6], A[7], I(0), A[8], I(0), A[9], Z(HUGE), None)
    take(f"topk_distill_backward {n}x{v}x{d}:{t}", st)
'''


def test_largest_sizes_fit_their_launches(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    fake = str(tmp_path / "fake_hip.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "host", "fake_hip.cpp"), "-o", fake],
                   check=True, capture_output=True, text=True)
    res = subprocess.run([sys.executable, "-c", CHILD, LIB, fake], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    rows = [line.split() for line in res.stdout.splitlines()]
    assert len(rows) == 16 * 2 + 16 * 2 + 24 * 4
    bad = []
    for name, size, status, launches, empty, threads, groups, block, yz in rows:
        launches, empty, threads, groups, block, yz = map(int, (launches, empty, threads, groups, block, yz))
        if int(status) or not launches or empty or threads >= 1 << 32 or groups >= 1 << 32 or block > 1024 or yz > 65535:
            bad.append((name, size, status, launches, empty, threads, groups, block, yz))
    assert not bad, bad
