"""Embedding lookup and gradient against the 64-bit form, within the bounds derived
in operators_ref.py (forward: one fp32 product and one rounding)."""
import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, pad, offset=0):
    """t's values in rows `pad` elements longer, starting `offset` elements into a
    buffer whose other elements are 77."""
    buf = torch.full((t.shape[0] * (t.shape[1] + pad) + offset + 8,), 77.0, device=t.device, dtype=t.dtype)
    v = buf[offset:offset + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v, buf


def untouched(view, buf):
    """Every element of buf outside the view still holds 77."""
    n = int((buf == 77.0).sum())
    return n >= buf.numel() - view.numel()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (8, 100, 4096), (7, 33, 7), (300, 1000, 96), (2049, 50, 65), (5, 9, 2050)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_lookup(gpu, dtype, n, vocab, dim, pad, offset):
    g = gen(n + dim)
    W, _ = strided(rand(g, (vocab, dim), dtype), pad, offset)
    tokens = torch.randint(-2, vocab + 2, (n,), generator=g, device="cuda")
    out, buf = strided(torch.zeros(n, dim, device="cuda", dtype=dtype), pad, offset)
    scale = 1.7
    got = mo.embedding_forward(tokens, W, scale=scale, out=out)
    torch.cuda.synchronize()
    want = R.embed(tokens, W, torch.tensor(scale, dtype=F32).double().item())
    R.check(got, want, (R.U + R.ut(dtype)) * want.abs(), "Y")
    assert untouched(out, buf)


def test_lookup_does_not_read_past_the_matrix(gpu):
    """A padded token's row is zero even where the matrix holds NaN in row 0."""
    W = torch.full((4, 16), float("nan"), device="cuda")
    W[2] = 1.0
    Y = mo.embedding_forward(torch.tensor([-1, 4, 2, 1 << 40, -(1 << 62)], device="cuda"), W)
    torch.cuda.synchronize()
    assert bool((Y[[0, 1, 3, 4]] == 0).all()) and bool((Y[2] == 1).all())


def token_sets(kind, n, vocab, g):
    if kind == "uniform":
        return torch.randint(0, vocab, (n,), generator=g, device="cuda")
    if kind == "one":           # every position the same token: one run over every chunk
        return torch.full((n,), vocab - 1, device="cuda", dtype=torch.int64)
    if kind == "zipf":
        u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        return ((vocab + 1) ** u - 1).long().clamp(0, vocab - 1)
    if kind == "padded":        # half the positions padding, ids at both edges
        t = torch.randint(-vocab // 2, vocab + vocab // 2, (n,), generator=g, device="cuda")
        t[::5] = 0
        t[1::7] = vocab - 1
        return t
    if kind == "none":
        return torch.full((n,), -100, device="cuda", dtype=torch.int64)
    raise ValueError(kind)


@pytest.mark.parametrize("ydt,gdt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("kind", ["uniform", "one", "zipf", "padded", "none"])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (5, 3, 9), (64, 17, 2049), (1023, 700, 96), (9001, 300, 72), (4097, 40000, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(gpu, ydt, gdt, kind, n, vocab, dim, accumulate):
    g = gen(n * 7 + dim)
    tokens = token_sets(kind, n, vocab, g)
    dY, _ = strided(rand(g, (n, dim), ydt), 5 if n % 2 else 0, 1 if n % 2 else 0)
    old = rand(g, (vocab, dim), gdt)
    G, buf = strided(old, 3 if dim % 2 else 0, 1 if dim % 2 else 0)
    mo.embedding_backward(tokens, dY, G, scale=0.6, accumulate=accumulate)
    torch.cuda.synchronize()
    want, bound = R.embed_grad(tokens, dY, vocab, torch.tensor(0.6, dtype=F32).double().item())
    if accumulate:
        want = want + old.double()
        bound = bound + R.U * want.abs()
    R.check(G, want, bound + R.ut(gdt) * want.abs(), f"G {kind}")
    assert untouched(G, buf)
    if accumulate:
        named = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        named[tokens[(tokens >= 0) & (tokens < vocab)]] = True
        assert torch.equal(G[~named], old[~named])


def test_gradient_of_a_large_padded_batch(gpu):
    """Several sort tiles and digit passes, ids above 2^17, dY rows of the padding NaN."""
    g = gen(3)
    n, vocab, dim = 40000, 200001, 16
    tokens = token_sets("padded", n, vocab, g)
    dY = rand(g, (n, dim), BF)
    dY[(tokens < 0) | (tokens >= vocab)] = float("nan")
    G = torch.full((vocab, dim), float("nan"), device="cuda", dtype=F32)
    mo.embedding_backward(tokens, dY, G)
    torch.cuda.synchronize()
    want, bound = R.embed_grad(tokens, dY, vocab, 1.0)
    R.check(G, want, bound + R.U * want.abs(), "G")


def test_empty_batch_writes_zeros(gpu):
    G = torch.full((19, 33), 5.0, device="cuda")
    t, dY = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, 33, device="cuda")
    mo.embedding_backward(t, dY, G, accumulate=True)
    torch.cuda.synchronize()
    assert bool((G == 5).all())
    mo.embedding_backward(t, dY, G)
    torch.cuda.synchronize()
    assert bool((G == 0).all())
    assert mo.embedding_forward(t, G).shape == (0, 33)


@pytest.mark.parametrize("n,dim", [(3000, 2048), (700, 100)])
def test_gradient_is_reproducible(gpu, n, dim):
    g = gen(5)
    tokens = token_sets("zipf", n, 500, g)
    dY = rand(g, (n, dim), F32)
    a = mo.embedding_backward(tokens, dY, torch.empty(500, dim, device="cuda"))
    ws = torch.full((mo.embedding_workspace_bytes(n, 500, dim),), 255, dtype=torch.uint8, device="cuda")
    b = mo.embedding_backward(tokens, dY, torch.empty(500, dim, device="cuda"), workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
