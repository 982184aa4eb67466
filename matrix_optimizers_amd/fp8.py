"""Matrices in 8 bits: activations and weights as e4m3 numbers with a power-of-two scale
for each block of 128, their product, and a weight's gradient from an activation
kept in 8 bits (the calls of ``include/mo.h`` that begin with fp8).

A block of 128 neighbours of a row (for a weight of 128 x 128) is held as
``torch.float8_e4m3fn`` numbers q and one ``torch.float8_e8m0fnu`` scale 2^e, x = q 2^e,
with the least e >= -127 that leaves no element over 448.  Conventions (checks, outputs,
streams, workspaces, autograd) as in ``operators``.
"""
from __future__ import annotations

import ctypes
from typing import Tuple

import torch

from ._binding import MoFp8Matrix, _check, load_library
from .operators import _DTYPE, FP8, FP8_BLOCK, FP8_SCALE, _code, _device, _matrix, _On, _ptr


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _operand(q, scales, what: str, square=None) -> MoFp8Matrix:
    """square: whether the scales are of blocks of 128 x 128; None: by their rows."""
    ldq = _matrix(q, what, None, None, FP8)
    rows, cols = q.shape
    shape = scales.shape
    if square is None:
        square = len(shape) == 2 and shape[0] != rows
    srows, scols = -(-rows // FP8_BLOCK) if square else rows, -(-cols // FP8_BLOCK)
    lds, inc = 1, 0
    if len(shape) == 2 and shape[1] > 1 and scales.stride(1) != 1:   # by columns: others' transpose
        inc = _matrix(scales.t(), f"{what}'s scales, transposed,", scols, srows, FP8_SCALE)
    else:
        lds = _matrix(scales, what + "'s scales", srows, scols, FP8_SCALE)
    return MoFp8Matrix(_ptr(q), _ptr(scales), rows, ldq, lds, inc, FP8_BLOCK if square else 1)


def fp8_quantize(X, *, q=None, scales=None, stream=None) -> Tuple:
    """(q, scales) of X (rows, cols), float32 or bfloat16: q (rows, cols), scales (rows,
    ceil(cols / 128)).  An operand of fp8_matmul, or an activation kept for the backward
    pass.  An infinity or NaN takes no part in its block's scale and becomes NaN."""
    lib = load_library()
    dev = _device(X, q, scales)
    ldx = _matrix(X, "X")
    rows, cols = X.shape
    code = _code(X, "X")
    with _On(dev, stream) as on:
        q, ldq = on.matrix(q, "q", rows, cols, FP8)
        scales, lds = on.matrix(scales, "scales", rows, _blocks(cols), FP8_SCALE)
        _check(lib.fp8_quantize(_ptr(X), ldx, code, rows, cols, _ptr(q), ldq, _ptr(scales), lds, on.handle),
               "fp8_quantize")
    return q, scales


def fp8_dequantize(q, scales, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values of fp8_quantize's q and scales in float32 or bfloat16 (``out``'s dtype where
    it is given): exact in float32; in bfloat16 those under 2^-130 are rounded to multiples
    of 2^-133, and those over its largest are infinite."""
    lib = load_library()
    dev = _device(q, scales, out)
    ldq = _matrix(q, "q", dtype=FP8)
    rows, cols = q.shape
    lds = _matrix(scales, "scales", rows, _blocks(cols), FP8_SCALE)
    with _On(dev, stream) as on:
        out, ldx = _out(on, out, "out", rows, cols, dtype)
        _check(lib.fp8_dequantize(_ptr(q), ldq, _ptr(scales), lds, rows, cols, _ptr(out), ldx, _code(out, "out"),
                                  on.handle), "fp8_dequantize")
    return out


def _out(on, out, what, rows, cols, dtype):
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPE:
        raise TypeError(f"{what}: unsupported dtype {dtype} (float32 or bfloat16)")
    return on.matrix(out, what, rows, cols, dtype)


def fp8_quantize_weight(W, *, q=None, scales=None, qt=None, scales_t=None, need_t: bool = True, stream=None) -> Tuple:
    """(q, scales, qt, scales_t) of a weight W (rows, cols) in blocks of 128 x 128, and of its
    transpose: the same numbers, for the product with an output's gradient.  Without
    ``need_t`` the last two are None."""
    lib = load_library()
    dev = _device(W, q, scales, qt, scales_t)
    ldw = _matrix(W, "W")
    rows, cols = W.shape
    code = _code(W, "W")
    with _On(dev, stream) as on:
        q, ldq = on.matrix(q, "q", rows, cols, FP8)
        scales, lds = on.matrix(scales, "scales", _blocks(rows), _blocks(cols), FP8_SCALE)
        ldqt = ldst = 0
        if need_t:
            qt, ldqt = on.matrix(qt, "qt", cols, rows, FP8)
            scales_t, ldst = on.matrix(scales_t, "scales_t", _blocks(cols), _blocks(rows), FP8_SCALE)
        else:
            qt = scales_t = None
        _check(lib.fp8_quantize_weight(_ptr(W), ldw, code, rows, cols, _ptr(q), ldq, _ptr(scales), lds, _ptr(qt), ldqt,
                                       _ptr(scales_t), ldst, on.handle), "fp8_quantize_weight")
    return q, scales, qt, scales_t


def _matmul_args(A, a_scales, B, b_scales):
    a, b = _operand(A, a_scales, "A"), _operand(B, b_scales, "B")
    if A.shape[1] != B.shape[1]:
        raise ValueError(f"A and B must have the same columns, not {A.shape[1]} and {B.shape[1]}")
    return a, b


def _matmul_bytes(a, b, dim, code) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().fp8_matmul_workspace_bytes(a, b, dim, code, out),
           "fp8_matmul_workspace_bytes")
    return int(out.value)


def fp8_matmul_workspace_bytes(A, a_scales, B, b_scales, *, dtype=torch.bfloat16) -> int:
    """Workspace of fp8_matmul on these tensors with a result of this dtype."""
    a, b = _matmul_args(A, a_scales, B, b_scales)
    if dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return _matmul_bytes(a, b, A.shape[1], _DTYPE[dtype])


def fp8_matmul(A, a_scales, B, b_scales, *, dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """Y = A B^T (rows of A, rows of B) of two matrices in 8 bits: A (tokens, dim) of
    fp8_quantize or rms_norm_quantize, B a weight of fp8_quantize_weight, or either the other
    kind (scales with one row per row, or per 128 of them).  bfloat16, or ``out``'s dtype: see
    fp8_matmul in include/mo.h for the accuracy of the sums in each."""
    lib = load_library()
    dev = _device(A, a_scales, B, b_scales, out)
    a, b = _matmul_args(A, a_scales, B, b_scales)
    dim = A.shape[1]
    with _On(dev, stream) as on:
        out, ldy = _out(on, out, "out", a.rows, b.rows, dtype)
        code = _DTYPE[out.dtype]
        need = _matmul_bytes(a, b, dim, code) if workspace is None else 0
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.fp8_matmul(a, b, dim, _ptr(out), ldy, code, ws, have, on.handle), "fp8_matmul")
        del keep
    return out


def _wgrad_bytes(dY, ldy, ycode, x, dim, rows) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().fp8_weight_grad_workspace_bytes(_ptr(dY), ldy, ycode, x, dim, rows, out),
           "fp8_weight_grad_workspace_bytes")
    return int(out.value)


def fp8_weight_grad_workspace_bytes(dY, q, scales) -> int:
    """Workspace of fp8_weight_grad on these tensors."""
    x = _operand(q, scales, "q", square=False)
    ldy = _matrix(dY, "dY", rows=q.shape[0])
    return _wgrad_bytes(dY, ldy, _code(dY, "dY"), x, q.shape[1], dY.shape[1])


def fp8_weight_grad(dY, q, scales, G, *, accumulate: bool = False, workspace=None, stream=None):
    """G = dY^T X, the gradient of Y = X W^T for W (rows, dim), from the output's gradient dY
    (tokens, rows), float32 or bfloat16, and X (tokens, dim) as fp8_quantize or
    rms_norm_quantize kept it, into G, float32 or bfloat16, the one that an owner step
    reads; with ``accumulate`` it is added to G.  Returns G."""
    lib = load_library()
    dev = _device(dY, q, scales, G)
    x = _operand(q, scales, "q", square=False)
    tokens, dim = q.shape
    ldy = _matrix(dY, "dY", rows=tokens)
    rows = dY.shape[1]
    ldg = _matrix(G, "G", rows, dim)
    ycode, gcode = _code(dY, "dY"), _code(G, "G")
    with _On(dev, stream) as on:
        need = _wgrad_bytes(dY, ldy, ycode, x, dim, rows) if workspace is None else 0
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.fp8_weight_grad(_ptr(dY), ldy, ycode, x, dim, _ptr(G), ldg, gcode, rows,
                                   1 if accumulate else 0, ws, have, on.handle), "fp8_weight_grad")
        del keep
    return G
