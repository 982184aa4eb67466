"""The embedding, layer norm and output-head entry points on the CPU: every check
returns its status before anything is enqueued (no call here reaches the HIP
runtime), the workspace sizes, and the binding's own refusals."""
import ctypes
import math

import pytest
import torch

import matrix_optimizers_amd as mo
from matrix_optimizers_amd import _binding as B

OK, INVALID, UNSUPPORTED, WS_SMALL, ALIAS = 0, -1, -2, -3, -4
GiB = 1 << 30
BASE = 1 << 44
A = [BASE + 64 * k * GiB for k in range(16)]   # addresses far apart
HUGE = 1 << 45


def size_of(fn, *args):
    out = ctypes.c_size_t(123)
    st = fn(*args, ctypes.byref(out))
    return st, out.value


# ---- embedding ---------------------------------------------------------------------

def emb_fwd(tokens=A[0], n=10, W=A[1], ld_w=0, vocab=100, dim=64, dtype=1, scale=1.0, Y=A[2], ld_y=0):
    return mo.load_library().embedding_forward(tokens, n, W, ld_w, vocab, dim, dtype, scale, Y, ld_y, None)


def emb_bwd(tokens=A[0], n=10, dY=A[1], ld_dy=0, dyt=1, G=A[2], ld_g=0, gt=1, vocab=100, dim=64, scale=1.0, acc=0,
            ws=A[3], have=HUGE):
    return mo.load_library().embedding_backward(tokens, n, dY, ld_dy, dyt, G, ld_g, gt, vocab, dim, scale, acc, ws,
                                                have, None)


def test_embedding_noops():
    assert emb_fwd(n=0) == OK and emb_fwd(dim=0) == OK and emb_fwd(n=0, tokens=None, Y=None, W=None) == OK
    assert emb_bwd(n=0, acc=1, G=None) == OK and emb_bwd(vocab=0, G=None) == OK and emb_bwd(dim=0) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=None), INVALID), (dict(W=None), INVALID), (dict(Y=None), INVALID), (dict(n=-1), INVALID),
    (dict(vocab=-1), INVALID), (dict(dim=-1), INVALID), (dict(ld_w=63), INVALID), (dict(ld_y=63), INVALID),
    (dict(ld_w=-1), INVALID), (dict(ld_w=(1 << 26) + 1), UNSUPPORTED), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(n=(1 << 30) + 1), UNSUPPORTED),
    (dict(vocab=(1 << 27) + 1), UNSUPPORTED), (dict(dim=(1 << 20) + 1), UNSUPPORTED),
    (dict(Y=A[1] + 128), ALIAS), (dict(Y=A[0] + 8), ALIAS)])
def test_embedding_forward_refusals(kw, code):
    assert emb_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=None), INVALID), (dict(dY=None), INVALID), (dict(G=None), INVALID), (dict(n=-1), INVALID),
    (dict(ld_dy=63), INVALID), (dict(ld_g=10), INVALID), (dict(scale=math.nan), INVALID), (dict(dyt=7), UNSUPPORTED),
    (dict(gt=-1), UNSUPPORTED), (dict(ws=None), WS_SMALL), (dict(have=100), WS_SMALL), (dict(G=A[1] + 64), ALIAS),
    (dict(ws=A[2] + 64), ALIAS), (dict(G=A[0]), ALIAS), (dict(vocab=(1 << 27) + 1), UNSUPPORTED)])
def test_embedding_backward_refusals(kw, code):
    assert emb_bwd(**kw) == code


def test_embedding_workspace():
    lib = mo.load_library()
    st, need = size_of(lib.embedding_workspace_bytes, 10, 100, 64)
    # keys and positions twice, the counts, two fp32 rows per chunk of positions
    assert st == OK and need >= 4 * 10 * 4 + 128 * 4 + 2 * 3 * 64 * 4
    assert emb_bwd(have=need - 1) == WS_SMALL
    for empty in ((0, 100, 64), (10, 0, 64), (10, 100, 0)):
        assert size_of(lib.embedding_workspace_bytes, *empty) == (OK, 0)
    assert size_of(lib.embedding_workspace_bytes, -1, 1, 1)[0] == INVALID
    assert lib.embedding_workspace_bytes(1, 1, 1, None) == INVALID
    # grows with the positions and the row, not with the vocabulary
    assert mo.embedding_workspace_bytes(16384, 128256, 4096) < 80 << 20


# ---- layer norm --------------------------------------------------------------------

def ln_fwd(X=A[0], ldx=0, w=A[1], b=A[2], Y=A[3], ldy=0, mean=A[4], rstd=A[5], rows=10, cols=64, dtype=1, eps=1e-5):
    return mo.load_library().layer_norm_forward(X, ldx, w, b, Y, ldy, mean, rstd, rows, cols, dtype, eps, None)


def ln_bwd(dY=A[0], lddy=0, X=A[1], ldx=0, w=A[2], mean=A[3], rstd=A[4], dX=A[5], lddx=0, dw=A[6], db=A[7], rows=10,
           cols=64, dtype=1, ws=A[8], have=HUGE):
    return mo.load_library().layer_norm_backward(dY, lddy, X, ldx, w, mean, rstd, dX, lddx, dw, db, rows, cols, dtype,
                                                 ws, have, None)


def test_layer_norm_noops():
    assert ln_fwd(rows=0, X=None, Y=None) == OK and ln_fwd(cols=0) == OK
    assert ln_bwd(cols=0) == OK and ln_bwd(dX=None, dw=None, db=None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=1), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(cols=(1 << 24) + 1), UNSUPPORTED),
    (dict(rows=(1 << 32) + 1), UNSUPPORTED), (dict(Y=A[0]), ALIAS), (dict(mean=A[3] + 4), ALIAS),
    (dict(rstd=A[4]), ALIAS), (dict(w=A[3]), ALIAS)])
def test_layer_norm_forward_refusals(kw, code):
    assert ln_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), INVALID), (dict(dY=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(lddy=3), INVALID), (dict(ldx=3), INVALID), (dict(lddx=3), INVALID), (dict(dtype=9), UNSUPPORTED),
    (dict(dX=A[1]), ALIAS), (dict(dw=A[7] + 4), ALIAS), (dict(dw=A[2]), ALIAS), (dict(ws=A[5]), ALIAS),
    (dict(ws=None), WS_SMALL), (dict(have=64), WS_SMALL)])
def test_layer_norm_backward_refusals(kw, code):
    assert ln_bwd(**kw) == code


def test_layer_norm_workspace():
    lib = mo.load_library()
    st, need = size_of(lib.layer_norm_workspace_bytes, 10, 64)
    assert st == OK and need >= 2 * 64 * 4 and ln_bwd(have=need - 1) == WS_SMALL
    assert size_of(lib.layer_norm_workspace_bytes, 0, 64) == (OK, 0)
    assert lib.layer_norm_workspace_bytes(1, 1, None) == INVALID


# ---- output head -------------------------------------------------------------------

def head(**kw):
    d = dict(H=A[0], W=A[1], tokens=10, vocab=100, dim=64, ld_h=0, ld_w=0, dtype=1)
    d.update(kw)
    return B.MoHead(**d)


def topk(**kw):
    d = dict(ids=A[2], logits=A[3], ld_ids=0, ld_logits=0, k=4, dtype=0, temperature=1.0)
    d.update(kw)
    return B.MoTopk(**d)


def x_fwd(h=None, labels=A[2], loss=A[4], lse=A[5], ws=A[9], have=HUGE):
    h = h or head()
    return mo.load_library().softmax_xent_forward(ctypes.byref(h), labels, loss, lse, ws, have, None)


def x_bwd(h=None, labels=A[2], loss=A[4], lse=A[5], dloss=A[6], dH=A[7], ldh=0, dW=A[8], ldw=0, ws=A[9], have=HUGE):
    h = h or head()
    return mo.load_library().softmax_xent_backward(ctypes.byref(h), labels, loss, lse, dloss, dH, ldh, dW, ldw, ws,
                                                   have, None)


def d_fwd(h=None, t=None, loss=A[4], lse=A[5], z=A[6], ws=A[9], have=HUGE):
    h, t = h or head(), t or topk()
    return mo.load_library().topk_distill_forward(ctypes.byref(h), ctypes.byref(t), loss, lse, z, ws, have, None)


def d_bwd(h=None, t=None, lse=A[5], z=A[6], dloss=A[4], dH=A[7], ldh=0, dW=A[8], ldw=0, ws=A[9], have=HUGE):
    h, t = h or head(), t or topk()
    return mo.load_library().topk_distill_backward(ctypes.byref(h), ctypes.byref(t), lse, z, dloss, dH, ldh, dW, ldw,
                                                   ws, have, None)


BAD_HEADS = [(dict(tokens=-1), INVALID), (dict(vocab=0), INVALID), (dict(dim=0), INVALID), (dict(ld_h=63), INVALID),
             (dict(ld_w=2), INVALID), (dict(ld_h=-5), INVALID), (dict(dtype=3), UNSUPPORTED),
             (dict(tokens=(1 << 20) + 1), UNSUPPORTED), (dict(vocab=(1 << 26) + 1), UNSUPPORTED),
             (dict(dim=(1 << 16) + 1), UNSUPPORTED), (dict(H=None), INVALID), (dict(W=None), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_HEADS)
def test_head_refusals(kw, code):
    for call in (x_fwd, x_bwd, d_fwd, d_bwd):
        assert call(head(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), INVALID), (dict(k=1025), UNSUPPORTED), (dict(temperature=0.0), INVALID),
    (dict(temperature=-1.0), INVALID), (dict(temperature=math.nan), INVALID), (dict(temperature=1e30), INVALID),
    (dict(temperature=1e-42), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(ld_ids=3), INVALID),
    (dict(ld_logits=3), INVALID), (dict(ids=None), INVALID), (dict(logits=None), INVALID)])
def test_teacher_refusals(kw, code):
    for call in (d_fwd, d_bwd):
        assert call(t=topk(**kw)) == code


def test_head_noops_and_null_arguments():
    lib = mo.load_library()
    assert x_fwd(head(tokens=0)) == OK and d_fwd(head(tokens=0)) == OK
    assert x_bwd(dH=None, dW=None) == OK and x_bwd(head(tokens=0), dW=None) == OK
    assert lib.softmax_xent_forward(None, A[2], A[4], A[5], None, 0, None) == INVALID
    h = head()
    assert lib.topk_distill_forward(ctypes.byref(h), None, A[4], A[5], A[6], A[9], HUGE, None) == INVALID
    for kw in (dict(labels=None), dict(loss=None), dict(lse=None)):
        assert x_fwd(**kw) == INVALID and x_bwd(**kw) == INVALID
    assert x_bwd(dloss=None) == INVALID and d_fwd(z=None) == INVALID and d_bwd(z=None) == INVALID
    assert x_bwd(ldh=63) == INVALID and x_bwd(ldw=63) == INVALID


def test_head_aliases_and_workspaces():
    lib = mo.load_library()
    assert x_fwd(loss=A[5]) == ALIAS and x_fwd(lse=A[0] + 4) == ALIAS and x_fwd(ws=A[1]) == ALIAS
    assert x_bwd(dW=A[1]) == ALIAS and x_bwd(dH=A[0]) == ALIAS and x_bwd(dH=A[8] + 64) == ALIAS
    assert d_fwd(z=A[3]) == ALIAS and d_bwd(dH=A[6]) == ALIAS
    h = head()
    for back, call in ((0, x_fwd), (1, x_bwd)):
        st, need = size_of(lib.softmax_xent_workspace_bytes, ctypes.byref(h), back)
        assert st == OK and call(have=need - 1) == WS_SMALL and call(ws=None) == WS_SMALL
    t = topk()
    for back, call in ((0, d_fwd), (1, d_bwd)):
        st, need = size_of(lib.topk_distill_workspace_bytes, ctypes.byref(h), ctypes.byref(t), back)
        assert st == OK and call(have=need - 1) == WS_SMALL
    assert lib.softmax_xent_workspace_bytes(ctypes.byref(h), 0, None) == INVALID


def bytes_of(back, **kw):
    h = head(**kw)
    return size_of(mo.load_library().softmax_xent_workspace_bytes, ctypes.byref(h), back)[1]


def test_the_logits_are_never_kept():
    """Workspaces at 8192 tokens x 128256 x 4096: far below one bf16 copy of the
    logits (2.1 GB) forward, and bounded backward (a vocabulary four times as
    long takes no more)."""
    big = dict(tokens=8192, vocab=128256, dim=4096)
    assert bytes_of(0, **big) < 40 << 20
    assert bytes_of(1, **big) < 1900 << 20
    assert bytes_of(1, tokens=8192, vocab=4 * 128256, dim=4096) < 1900 << 20
    # a misaligned or strided head is copied in pieces, not whole
    assert bytes_of(0, W=A[1] + 2, **big) < 500 << 20


# ---- the binding's checks --------------------------------------------------------------

def test_binding_refuses_host_tensors_and_wrong_shapes():
    X, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: mo.embedding_forward(t, X), lambda: mo.embedding_backward(t, X, X.clone()),
                 lambda: mo.layer_norm_forward(X), lambda: mo.layer_norm_backward(X, X, X[:, 0], X[:, 0]),
                 lambda: mo.softmax_xent_forward(X, X, t), lambda: mo.topk_distill_forward(X, X, t[:, None], X[:, :1])):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_binding_matrix_checks():
    from matrix_optimizers_amd import operators as O
    x = torch.zeros(6, 8)
    assert O._matrix(x, "x") == 8 and O._matrix(x[:, 2:5], "x") == 8 and O._matrix(x[:1], "x") == 0
    assert O._matrix(x[::2], "x") == 16 and O._matrix(torch.zeros(0, 4), "x") == 0
    for bad in (x.t(), x[0].expand(6, 8), torch.zeros(2, 3, 4), torch.zeros(8)):
        with pytest.raises(ValueError):
            O._matrix(bad, "x")
    with pytest.raises(ValueError):
        O._matrix(x, "x", 6, 7)
    with pytest.raises(TypeError):
        O._matrix(x, "x", dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        O._code(x.half(), "x")
    with pytest.raises(ValueError):
        O._vector(x[:, 0], "v", 6)
    with pytest.raises(TypeError):
        O._vector(torch.zeros(3, dtype=torch.int32), "v", 3, torch.int64)


def test_operators_are_listed_and_lazy():
    import subprocess
    import sys
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys, matrix_optimizers_amd as mo\n"
            "assert 'torch' not in sys.modules\n"
            "assert 'embedding_forward' in dir(mo)\n"
            "mo.embedding_forward\n"
            "assert 'torch' in sys.modules\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    with pytest.raises(AttributeError):
        mo.no_such_operator
