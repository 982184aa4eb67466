"""Launches of the RMS norm and the 8-bit operators at the largest sizes the entry points
accept stay inside one launch's limits, as test_launch_limits does it for the others:
against a stand-in for the runtime's launches; the addresses are never used."""
import os
import shutil
import subprocess
import sys

import pytest

from test_launch_limits import HERE, LIB

CHILD = r'''
import ctypes, itertools, sys
fake = ctypes.CDLL(sys.argv[2], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[1])
P, I, N, F, Z = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t

class Mat(ctypes.Structure):
    _fields_ = [("q", P), ("scales", P), ("rows", I), ("ld_q", I), ("ld_scales", I), ("inc_scales", I), ("block_rows", N)]

HUGE = 1 << 59
A = [P(k << 59) for k in range(1, 31)]
def take(what, st):
    out = (ctypes.c_uint64 * 6)()
    fake.fake_hip_take(out)
    print(what, st, *out, flush=True)

edges = lambda *axes: itertools.product(*axes)
for r, c, t in edges((1, 1 << 27, 1 << 32), (1, 128, 1000, 1024, 4096, 8192, 16384, 16385, 1 << 24), (0, 1)):
    st = lib.rms_norm_forward(A[0], I(0), A[1], I(0), A[2], A[3], I(0), A[4], I(0), A[5], I(0), A[6], I(0), A[7], I(r), I(c),
                              N(t), F(1e-6), None)
    take(f"rms_norm_forward {r}x{c}:{t}", st)
    st = lib.rms_norm_backward(A[0], I(0), A[1], I(0), A[2], A[3], A[4], I(0), A[5], I(0), A[6], I(r), I(c), N(t), A[8],
                               Z(HUGE), None)
    take(f"rms_norm_backward {r}x{c}:{t}", st)
    st = lib.fp8_quantize(A[0], I(0), N(t), I(r), I(c), A[1], I(0), A[2], I(0), None)
    take(f"fp8_quantize {r}x{c}:{t}", st)
    st = lib.fp8_dequantize(A[0], I(0), A[1], I(0), I(r), I(c), A[2], I(0), N(t), None)
    take(f"fp8_dequantize {r}x{c}:{t}", st)
S = 1 << 20
for r, c, t in edges((1, 129, S), (1, 129, S), (0, 1)):
    st = lib.fp8_quantize_weight(A[0], I(0), N(t), I(r), I(c), A[1], I(0), A[2], I(0), A[3], I(0), A[4], I(0), None)
    take(f"fp8_quantize_weight {r}x{c}:{t}", st)
# every way of reading: in place, scales copied, converted, a few rows
for m, n, k, t, pad, inc, blk in edges((1, 33, 65, 4097, S), (1, 4097, S), (1, 512, S), (0, 1), (0, 1), (0, 1), (1, 128)):
    kb = (k + 127) // 128
    srows = m if blk == 1 else (m + 127) // 128
    a = Mat(A[0], A[1], m, k + pad, 1 if inc and srows > 1 and kb > 1 else 0, srows if inc and srows > 1 and kb > 1 else 0, blk)
    b = Mat(A[2], A[3], n, 0, 0, 0, 128)
    st = lib.fp8_matmul(ctypes.byref(a), ctypes.byref(b), I(k), A[4], I(0), N(t), A[5], Z(HUGE), None)
    take(f"fp8_matmul {m}x{n}x{k}:{t},{pad},{inc},{blk}", st)
for m, n, k, t, pad in edges((1, 4097, S), (8, 4097, S), (16, 4097, S), (0, 1), (0, 1)):
    x = Mat(A[2], A[3], m, k + pad, 0, 0, 1)
    st = lib.fp8_weight_grad(A[0], I(0), N(t), ctypes.byref(x), I(k), A[4], I(0), N(t), I(n), N(pad), A[5], Z(HUGE), None)
    take(f"fp8_weight_grad {m}x{n}x{k}:{t},{pad}", st)
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
    assert len(rows) == 54 * 4 + 18 + 720 + 108
    bad = []
    for name, size, status, launches, empty, threads, groups, block, yz in rows:
        launches, empty, threads, groups, block, yz = map(int, (launches, empty, threads, groups, block, yz))
        if int(status) or not launches or empty or threads >= 1 << 32 or groups >= 1 << 32 or block > 1024 or yz > 65535:
            bad.append((name, size, status, launches, empty, threads, groups, block, yz))
    assert not bad, bad[:20]
