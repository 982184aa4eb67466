"""The operators that write the gradients the owner steps read: the embedding, the
layer norm, the RMS norm, the softmax cross entropy of the output head and distillation
from a teacher's top logits (the second half of ``include/mo.h``; matrices in 8 bits
are in ``fp8``).

Argument marshalling only, as in ``_binding``: tensors are checked, outputs the
caller does not pass are allocated (on the launch stream), and the call runs in
the library's HIP kernels on the tensors' device, on ``stream`` or that device's
current stream.  Nothing is registered with autograd: a backward pass is the call
that computes it, and what a call returns has no grad_fn, also where an input requires
gradients.  Layers that autograd runs between two calls start from a result marked
with ``requires_grad_()`` and are driven by ``h.backward(dh)`` with the gradient the
next call computed; the first one's gradient is then that result's ``.grad``.  A caller's workspace (a uint8 tensor of at least the
``*_workspace_bytes`` figure) must not be reused by other work before the call has
finished on its stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _binding as B
from ._binding import MoHead, MoTopk, _check, load_library

TOPK_MAX = 1024   # MO_TOPK_MAX of include/mo.h
FP8_BLOCK = 128   # MO_FP8_BLOCK
FP8, FP8_SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu

_DTYPE = {torch.float32: B.MO_F32, torch.bfloat16: B.MO_BF16}
_empty = torch.empty


# ---------------------------------------------------------------------------
# checks, allocation, streams
# ---------------------------------------------------------------------------

def _device(*tensors):
    """The one HIP device of the tensors (None entries are skipped)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
            if dev.type != "cuda":
                raise ValueError("tensors must be on a HIP device")
        elif t.device != dev:
            raise ValueError("tensors must be on one device")
    return dev


def _code(t, what: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _matrix(t, what: str, rows: Optional[int] = None, cols: Optional[int] = None, dtype=None) -> int:
    """Checks a row-major matrix; its row stride in elements."""
    shape = t.shape
    if len(shape) == 2:
        r, c = shape
        if (rows is None or r == rows) and (cols is None or c == cols) and (dtype is None or t.dtype is dtype):
            if not r or not c:
                return 0
            s0, s1 = t.stride()
            if s1 == 1 or c == 1:
                if r == 1:
                    return 0
                if s0 >= c:
                    return s0
    return _not_a_matrix(t, what, rows, cols, dtype)


def _not_a_matrix(t, what, rows, cols, dtype) -> int:
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        want = f"({'rows' if rows is None else rows}, {'cols' if cols is None else cols})"
        raise ValueError(f"{what} must be 2D {want}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must be row-major with unit column stride")
    # a row stride of 0 (an expanded row) or less than a row would alias rows
    raise ValueError(f"{what} has overlapping rows (stride {t.stride(0)})")


def _vector(t, what: str, n: int, dtype=torch.float32) -> None:
    shape = t.shape
    if len(shape) != 1 or shape[0] != n:
        raise ValueError(f"{what} must be a vector of {n}, not {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")


def _ptr(t):
    return t.data_ptr() or None if t is not None else None


class _On:
    """The device and stream of one call: makes the tensors' device current, and
    allocates with the launch stream current (so that the caching allocator
    hands a freed block out again only in that stream's order)."""

    __slots__ = ("dev", "stream", "guards", "handle")

    def __init__(self, dev, stream):
        self.dev, self.stream, self.guards = dev, stream, ()

    def __enter__(self):
        try:
            return self._enter()
        except BaseException:
            self.__exit__()   # a with statement would not
            raise

    def _enter(self):
        dev, stream = self.dev, self.stream
        if torch.cuda.current_device() != dev.index:
            self._guard(torch.cuda.device(dev))
        if stream is None:
            # the handle alone: building a Stream object costs as much as the rest of a small call
            self.handle = torch._C._cuda_getCurrentRawStream(dev.index)
            return self
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(B._stream_handle(stream), device=dev)
        elif stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
        self.handle = stream.cuda_stream
        self._guard(torch.cuda.stream(stream))
        return self

    def _guard(self, g):
        g.__enter__()
        self.guards += (g,)

    def __exit__(self, *exc):
        while self.guards:
            g, self.guards = self.guards[-1], self.guards[:-1]
            g.__exit__(None, None, None)

    def matrix(self, t, what, rows, cols, dtype):
        """(t, row stride): the caller's matrix, checked, or a new one."""
        if t is None:
            return _empty(rows, cols, dtype=dtype, device=self.dev), 0
        return t, _matrix(t, what, rows, cols, dtype)

    def vector(self, t, what, n):
        if t is None:
            return _empty(n, dtype=torch.float32, device=self.dev)
        _vector(t, what, n)
        return t

    def workspace(self, workspace, need: int):
        """(address, bytes, the tensor to keep until the launch)."""
        if workspace is None:
            if need == 0:
                return None, 0, None
            workspace = torch.empty(need, dtype=torch.uint8, device=self.dev)
        elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != self.dev:
            raise ValueError("workspace must be a contiguous uint8 tensor on the tensors' device")
        return workspace.data_ptr(), workspace.numel(), workspace


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

def embedding_forward(tokens, W, *, scale: float = 1.0, out=None, stream=None):
    """Y[i] = scale * W[tokens[i]]: tokens int64 (n,), W (vocab, dim) float32 or
    bfloat16, Y (n, dim) of W's dtype.  A token outside 0 .. vocab - 1 (padding)
    gives a zero row."""
    lib = load_library()
    dev = _device(tokens, W, out)
    n = tokens.numel()
    _vector(tokens, "tokens", n, torch.int64)
    ldw = _matrix(W, "W")
    vocab, dim = W.shape
    code = _code(W, "W")
    with _On(dev, stream) as on:
        out, ldy = on.matrix(out, "out", n, dim, W.dtype)
        _check(lib.embedding_forward(_ptr(tokens), n, _ptr(W), ldw, vocab, dim, code, scale, _ptr(out), ldy,
                                     on.handle), "embedding_forward")
    return out


def embedding_workspace_bytes(n: int, vocab: int, dim: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().embedding_workspace_bytes(n, vocab, dim, ctypes.byref(out)), "embedding_workspace_bytes")
    return int(out.value)


def embedding_backward(tokens, dY, G, *, scale: float = 1.0, accumulate: bool = False, workspace=None,
                       stream=None):
    """The lookup's gradient into G (vocab, dim), float32 or bfloat16, whose rows
    without a token become zero; with ``accumulate`` it is added to G and those
    rows stay (a matrix tied to the output head).  Returns G."""
    lib = load_library()
    dev = _device(tokens, dY, G)
    n = tokens.numel()
    _vector(tokens, "tokens", n, torch.int64)
    ldg = _matrix(G, "G")
    vocab, dim = G.shape
    ldy = _matrix(dY, "dY", n, dim)
    ycode, gcode = _code(dY, "dY"), _code(G, "G")
    need = embedding_workspace_bytes(n, vocab, dim)
    with _On(dev, stream) as on:
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.embedding_backward(_ptr(tokens), n, _ptr(dY), ldy, ycode, _ptr(G), ldg, gcode, vocab, dim, scale,
                                      1 if accumulate else 0, ws, have, on.handle), "embedding_backward")
        del keep
    return G


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def layer_norm_forward(X, weight=None, bias=None, *, eps: float = 1e-5, out=None, mean=None, rstd=None,
                       stream=None) -> Tuple:
    """(Y, mean, rstd) of the rows of X (rows, cols), float32 or bfloat16; weight and
    bias are float32 vectors (slices of the packed tail) or None.  Rows without
    elements have no mean: mean and rstd are NaN then."""
    lib = load_library()
    dev = _device(X, weight, bias, out, mean, rstd)
    ldx = _matrix(X, "X")
    rows, cols = X.shape
    code = _code(X, "X")
    if weight is not None:
        _vector(weight, "weight", cols)
    if bias is not None:
        _vector(bias, "bias", cols)
    with _On(dev, stream) as on:
        out, ldy = on.matrix(out, "out", rows, cols, X.dtype)
        mean, rstd = on.vector(mean, "mean", rows), on.vector(rstd, "rstd", rows)
        _check(lib.layer_norm_forward(_ptr(X), ldx, _ptr(weight), _ptr(bias), _ptr(out), ldy, _ptr(mean),
                                      _ptr(rstd), rows, cols, code, eps, on.handle), "layer_norm_forward")
        if cols == 0:   # the library writes nothing then
            mean.fill_(float("nan"))
            rstd.fill_(float("nan"))
    return out, mean, rstd


def layer_norm_workspace_bytes(rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().layer_norm_workspace_bytes(rows, cols, ctypes.byref(out)), "layer_norm_workspace_bytes")
    return int(out.value)


def layer_norm_backward(dY, X, mean, rstd, weight=None, *, dX=None, dweight=None, dbias=None,
                        need_dX: bool = True, need_dweight: bool = True, need_dbias: bool = True,
                        workspace=None, stream=None) -> Tuple:
    """(dX, dweight, dbias) from layer_norm_forward's X, mean, rstd and weight; dX of
    X's dtype, dweight and dbias float32 (slices of the tail's gradient).  The
    ones not needed are neither computed nor returned (None)."""
    lib = load_library()
    dev = _device(dY, X, mean, rstd, weight, dX, dweight, dbias)
    ldx = _matrix(X, "X")
    rows, cols = X.shape
    code = _code(X, "X")
    ldy = _matrix(dY, "dY", rows, cols, X.dtype)
    _vector(mean, "mean", rows)
    _vector(rstd, "rstd", rows)
    if weight is not None:
        _vector(weight, "weight", cols)
    need = layer_norm_workspace_bytes(rows, cols) if need_dweight or need_dbias else 0
    with _On(dev, stream) as on:
        dX, lddx = on.matrix(dX, "dX", rows, cols, X.dtype) if need_dX else (None, 0)
        out = (dX, on.vector(dweight, "dweight", cols) if need_dweight else None,
               on.vector(dbias, "dbias", cols) if need_dbias else None)
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.layer_norm_backward(_ptr(dY), ldy, _ptr(X), ldx, _ptr(weight), _ptr(mean), _ptr(rstd),
                                       _ptr(out[0]), lddx, _ptr(out[1]), _ptr(out[2]), rows, cols, code, ws, have,
                                       on.handle), "layer_norm_backward")
        del keep
    return out


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def _rms_forward(X, weight, residual, eps, out, q, scales, h, rstd, stream, to8: bool):
    lib = load_library()
    dev = _device(X, weight, residual, out, q, scales, h, rstd)
    ldx = _matrix(X, "X")
    rows, cols = X.shape
    code = _code(X, "X")
    if weight is not None:
        _vector(weight, "weight", cols)
    if residual is None and h is not None:
        raise ValueError("h is written where there is a residual; without one it is X")
    ldr = 0 if residual is None else _matrix(residual, "residual", rows, cols, X.dtype)
    with _On(dev, stream) as on:
        ldy = ldq = lds = ldh = 0
        if to8:
            q, ldq = on.matrix(q, "q", rows, cols, FP8)
            scales, lds = on.matrix(scales, "scales", rows, -(-cols // FP8_BLOCK), FP8_SCALE)
        else:
            out, ldy = on.matrix(out, "out", rows, cols, X.dtype)
        if residual is not None:
            h, ldh = on.matrix(h, "h", rows, cols, X.dtype)
        rstd = on.vector(rstd, "rstd", rows)
        _check(lib.rms_norm_forward(_ptr(X), ldx, _ptr(residual), ldr, _ptr(weight), _ptr(h), ldh, _ptr(out), ldy,
                                    _ptr(q), ldq, _ptr(scales), lds, _ptr(rstd), rows, cols, code, eps, on.handle),
               "rms_norm_forward")
        if cols == 0:   # the library writes nothing then
            rstd.fill_(float("nan"))
    return ((q, scales) if to8 else (out,)) + (X if residual is None else h, rstd)


def rms_norm_forward(X, weight=None, *, residual=None, eps: float = 1e-6, out=None, h=None, rstd=None,
                     stream=None) -> Tuple:
    """(Y, h, rstd) of the rows of h = X + residual (rows, cols), float32 or bfloat16,
    rounded to their type: Y = h * rstd * weight, rstd = (mean(h^2) + eps)^-1/2.  weight is a
    float32 vector (a slice of the packed tail) or None; without a residual h is X itself.
    Rows without elements have no rstd: it is NaN then."""
    return _rms_forward(X, weight, residual, eps, out, None, None, h, rstd, stream, False)


def rms_norm_quantize(X, weight=None, *, residual=None, eps: float = 1e-6, q=None, scales=None, h=None, rstd=None,
                      stream=None) -> Tuple:
    """(q, scales, h, rstd): as rms_norm_forward, with Y in 8 bits as fp8_quantize makes it,
    without a rounding to X's type before."""
    return _rms_forward(X, weight, residual, eps, None, q, scales, h, rstd, stream, True)


def rms_norm_workspace_bytes(rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().rms_norm_workspace_bytes(rows, cols, ctypes.byref(out)), "rms_norm_workspace_bytes")
    return int(out.value)


def rms_norm_backward(dY, h, rstd, weight=None, *, dH=None, dX=None, dweight=None, need_dX: bool = True,
                      need_dweight: bool = True, workspace=None, stream=None) -> Tuple:
    """(dX, dweight) from the forward call's h, rstd and weight; dX of h's dtype is the
    gradient of X and of the residual alike, dweight is float32 (a slice of the tail's
    gradient).  dH, the gradient that reaches h by other ways (down the residual
    stream), is added to dX.  The ones not needed are neither computed nor returned (None)."""
    lib = load_library()
    dev = _device(dY, h, rstd, weight, dH, dX, dweight)
    ldh = _matrix(h, "h")
    rows, cols = h.shape
    code = _code(h, "h")
    ldy = _matrix(dY, "dY", rows, cols, h.dtype)
    lddh = 0 if dH is None else _matrix(dH, "dH", rows, cols, h.dtype)
    _vector(rstd, "rstd", rows)
    if weight is not None:
        _vector(weight, "weight", cols)
    need = rms_norm_workspace_bytes(rows, cols) if need_dweight else 0
    with _On(dev, stream) as on:
        dX, lddx = on.matrix(dX, "dX", rows, cols, h.dtype) if need_dX else (None, 0)
        dweight = on.vector(dweight, "dweight", cols) if need_dweight else None
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.rms_norm_backward(_ptr(dY), ldy, _ptr(h), ldh, _ptr(weight), _ptr(rstd), _ptr(dH), lddh, _ptr(dX),
                                     lddx, _ptr(dweight), rows, cols, code, ws, have, on.handle), "rms_norm_backward")
        del keep
    return dX, dweight


# ---------------------------------------------------------------------------
# output head
# ---------------------------------------------------------------------------

def _head(H, W) -> MoHead:
    ldh, ldw = _matrix(H, "H"), _matrix(W, "W", cols=H.shape[1], dtype=H.dtype)
    return MoHead(H=_ptr(H), W=_ptr(W), tokens=H.shape[0], vocab=W.shape[0], dim=H.shape[1], ld_h=ldh, ld_w=ldw,
                  dtype=_code(H, "H"))


def _topk(H, ids, logits, temperature: float) -> MoTopk:
    ld_ids = _matrix(ids, "ids", rows=H.shape[0], dtype=torch.int64)
    k = ids.shape[1]
    ld_logits = _matrix(logits, "logits", H.shape[0], k)
    return MoTopk(ids=_ptr(ids), logits=_ptr(logits), ld_ids=ld_ids, ld_logits=ld_logits, k=k,
                  dtype=_code(logits, "logits"), temperature=temperature)


def softmax_xent_workspace_bytes(H, W, backward: bool = False) -> int:
    """Workspace of the forward or the backward call on these tensors."""
    out = ctypes.c_size_t(0)
    head = _head(H, W)
    _check(load_library().softmax_xent_workspace_bytes(ctypes.byref(head), 1 if backward else 0, ctypes.byref(out)),
           "softmax_xent_workspace_bytes")
    return int(out.value)


def topk_distill_workspace_bytes(H, W, ids, logits, *, temperature: float = 1.0, backward: bool = False) -> int:
    out = ctypes.c_size_t(0)
    head, top = _head(H, W), _topk(H, ids, logits, temperature)
    _check(load_library().topk_distill_workspace_bytes(ctypes.byref(head), ctypes.byref(top), 1 if backward else 0,
                                                       ctypes.byref(out)), "topk_distill_workspace_bytes")
    return int(out.value)


def softmax_xent_forward(H, W, labels, *, loss=None, lse=None, workspace=None, stream=None) -> Tuple:
    """(loss, lse), float32 per token, of the hidden states H (tokens, dim) under the
    head W (vocab, dim), both float32 or both bfloat16; the logits are not
    stored.  labels int64 (tokens,); one outside 0 .. vocab - 1 marks a position
    without a target, whose loss and lse are 0."""
    lib = load_library()
    dev = _device(H, W, labels, loss, lse)
    head = _head(H, W)
    n = H.shape[0]
    _vector(labels, "labels", n, torch.int64)
    with _On(dev, stream) as on:
        loss, lse = on.vector(loss, "loss", n), on.vector(lse, "lse", n)
        need = softmax_xent_workspace_bytes(H, W) if workspace is None else 0
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.softmax_xent_forward(ctypes.byref(head), _ptr(labels), _ptr(loss), _ptr(lse), ws, have,
                                        on.handle), "softmax_xent_forward")
        del keep
    return loss, lse


def _grads(on, H, W, dH, dW, need_dH, need_dW):
    dH, ldh = on.matrix(dH, "dH", H.shape[0], H.shape[1], H.dtype) if need_dH else (None, 0)
    dW, ldw = on.matrix(dW, "dW", W.shape[0], W.shape[1], W.dtype) if need_dW else (None, 0)
    return dH, ldh, dW, ldw


def softmax_xent_backward(H, W, labels, loss, lse, dloss, *, dH=None, dW=None, need_dH: bool = True,
                          need_dW: bool = True, workspace=None, stream=None) -> Tuple:
    """(dH, dW), of H's dtype, of sum(dloss * loss), from the forward call's loss and
    lse.  dloss float32 (tokens,): 1 / count for a mean; a row of 0 takes no part.
    dW may be the G that an owner step reads."""
    lib = load_library()
    dev = _device(H, W, labels, loss, lse, dloss, dH, dW)
    head = _head(H, W)
    n = H.shape[0]
    _vector(labels, "labels", n, torch.int64)
    for t, what in ((loss, "loss"), (lse, "lse"), (dloss, "dloss")):
        _vector(t, what, n)
    with _On(dev, stream) as on:
        dH, ldh, dW, ldw = _grads(on, H, W, dH, dW, need_dH, need_dW)
        need = softmax_xent_workspace_bytes(H, W, backward=True) if workspace is None else 0
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.softmax_xent_backward(ctypes.byref(head), _ptr(labels), _ptr(loss), _ptr(lse), _ptr(dloss),
                                         _ptr(dH), ldh, _ptr(dW), ldw, ws, have, on.handle), "softmax_xent_backward")
        del keep
    return dH, dW


def topk_distill_forward(H, W, ids, logits, *, temperature: float = 1.0, loss=None, lse=None, z=None,
                         workspace=None, stream=None) -> Tuple:
    """(loss, lse, z): the distillation loss T^2 KL(p || q) per token, p the softmax
    of a teacher's top logits (tokens, k), float32 or bfloat16, at the int64 ids
    (tokens, k), q the student's softmax over the whole vocabulary, both at
    temperature T.  Ids outside 0 .. vocab - 1 are absent entries; a row without
    any has loss 0.  lse and z (the student's logits at the ids) are for the
    backward call."""
    lib = load_library()
    dev = _device(H, W, ids, logits, loss, lse, z)
    head, top = _head(H, W), _topk(H, ids, logits, temperature)
    n, k = ids.shape
    with _On(dev, stream) as on:
        loss, lse = on.vector(loss, "loss", n), on.vector(lse, "lse", n)
        z, _ = on.matrix(z, "z", n, k, torch.float32)
        _contiguous(z)
        need = topk_distill_workspace_bytes(H, W, ids, logits, temperature=temperature) if workspace is None else 0
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.topk_distill_forward(ctypes.byref(head), ctypes.byref(top), _ptr(loss), _ptr(lse), _ptr(z), ws,
                                        have, on.handle), "topk_distill_forward")
        del keep
    return loss, lse, z


def _contiguous(z) -> None:
    if not z.is_contiguous():
        raise ValueError("z must be contiguous")


def topk_distill_backward(H, W, ids, logits, lse, z, dloss, *, temperature: float = 1.0, dH=None, dW=None,
                          need_dH: bool = True, need_dW: bool = True, workspace=None, stream=None) -> Tuple:
    """(dH, dW), of H's dtype, of sum(dloss * loss), from the forward call's lse and z."""
    lib = load_library()
    dev = _device(H, W, ids, logits, lse, z, dloss, dH, dW)
    head, top = _head(H, W), _topk(H, ids, logits, temperature)
    n, k = ids.shape
    _vector(lse, "lse", n)
    _vector(dloss, "dloss", n)
    _matrix(z, "z", n, k, torch.float32)
    _contiguous(z)
    with _On(dev, stream) as on:
        dH, ldh, dW, ldw = _grads(on, H, W, dH, dW, need_dH, need_dW)
        need = topk_distill_workspace_bytes(H, W, ids, logits, temperature=temperature, backward=True) \
            if workspace is None else 0
        ws, have, keep = on.workspace(workspace, need)
        _check(lib.topk_distill_backward(ctypes.byref(head), ctypes.byref(top), _ptr(lse), _ptr(z), _ptr(dloss),
                                         _ptr(dH), ldh, _ptr(dW), ldw, ws, have, on.handle), "topk_distill_backward")
        del keep
    return dH, dW
