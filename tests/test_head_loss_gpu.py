"""Softmax cross entropy and distillation over the output head against the 64-bit
forms, within the bounds derived in operators_ref.py."""
import math

import pytest
import torch

import matrix_optimizers_amd as mo
import operators_ref as R
from test_embedding_gpu import gen, rand, strided, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# tokens around the tile widths 64, 128, 256; vocabularies around a tile of 256 rows; row
# lengths that are whole stages in place, and ones that are copied (odd, 192, short)
SHAPES = [(1, 1, 1), (1, 1000, 64), (2, 255, 7), (37, 256, 64), (64, 257, 128), (65, 5, 96), (128, 1000, 192),
          (129, 2049, 256), (200, 511, 320), (257, 513, 100), (300, 3000, 576), (700, 300, 130)]


def inputs(n, vocab, dim, dtype, seed, pad=0):
    g = gen(seed)
    W, _ = strided(rand(g, (vocab, dim), dtype, 1 / math.sqrt(dim)), pad, pad // 2)
    H, _ = strided(rand(g, (n, dim), dtype, 2.0), pad, pad // 3)
    dloss = torch.randn(n, generator=g, device="cuda") / n
    if n > 2:
        dloss[1] = 0
    return g, H, W, dloss


def labels_of(g, n, vocab):
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    y[torch.rand(n, generator=g, device="cuda") < 0.2] = -100
    if n > 4:
        y[3], y[4] = vocab, vocab - 1
    return y


def teacher_of(g, n, vocab, k, dtype):
    ids = torch.randint(-max(1, vocab // 10), vocab + 1, (n, k), generator=g, device="cuda")
    t = (torch.randn((n, k), generator=g, device="cuda") * 3).to(dtype)
    t[(ids < 0) | (ids >= vocab)] = float("nan")      # absent entries hold anything
    if n > 5:
        ids[2] = -1                                    # no entry at all
        ids[3, : k // 2 + 1] = vocab - 1               # one id several times
        t[3, : k // 2 + 1] = 1.0
        t[4] = torch.where(torch.isnan(t[4]), t[4], torch.full_like(t[4], -math.inf))   # all weight gone
        t[5, 0], ids[5, 0] = torch.finfo(dtype).min, 0
    return ids, t


def compare(got, want, dH=None, dW=None):
    R.check(got[0], want["loss"], want["b_loss"], "loss")
    R.check(got[1], want["lse"], want["b_lse"], "lse")
    if dH is not None:
        R.check(dH, want["dH"], want["b_dH"], "dH")
        R.check(dW, want["dW"], want["b_dW"], "dW")


def run_xent(H, W, y, dloss, pad=0):
    """One step into strided outputs; checks what lies around them."""
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, bh = strided(torch.zeros_like(H), pad, pad // 2)
    dW, bw = strided(torch.zeros_like(W), pad, pad // 2)
    mo.softmax_xent_backward(H, W, y, loss, lse, dloss, dH=dH, dW=dW)
    torch.cuda.synchronize()
    assert untouched(dH, bh) and untouched(dW, bw)
    return (loss, lse), dH, dW


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,dim", SHAPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_cross_entropy(gpu, dtype, n, vocab, dim, pad):
    g, H, W, dloss = inputs(n, vocab, dim, dtype, n + vocab + dim, pad)
    y = labels_of(g, n, vocab)
    got, dH, dW = run_xent(H, W, y, dloss, pad)
    want = R.head(H, W, dloss, labels=y)
    compare(got, want, dH, dW)
    dead = ~want["live"]
    assert bool((got[0][dead] == 0).all()) and bool((got[1][dead] == 0).all()) and bool((dH[dead] == 0).all())


@pytest.mark.parametrize("dtype,tdt", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n,vocab,dim", SHAPES)
@pytest.mark.parametrize("k,T", [(1, 1.0), (10, 2.0), (130, 0.7)])
def test_distillation(gpu, dtype, tdt, n, vocab, dim, k, T):
    g, H, W, dloss = inputs(n, vocab, dim, dtype, n + vocab + dim + k)
    ids, t = teacher_of(g, n, vocab, k, tdt)
    T32 = torch.tensor(T, dtype=F32).double().item()
    loss, lse, z = mo.topk_distill_forward(H, W, ids, t, temperature=T)
    dH, dW = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss, temperature=T)
    torch.cuda.synchronize()
    clean = torch.where((ids >= 0) & (ids < vocab), t.double(), torch.zeros_like(t, dtype=torch.float64))
    want = R.head(H, W, dloss, ids=ids, teacher=clean, T=T32)
    compare((loss, lse), want, dH, dW)
    dead = ~want["live"]
    assert bool((loss[dead] == 0).all()) and bool((dH[dead] == 0).all())
    assert bool((z[(ids < 0) | (ids >= vocab)] == 0).all())


def test_strided_teacher_and_one_entry_is_cross_entropy(gpu):
    """A single stored entry at temperature 1 is the label: same loss and the same
    gradients as the cross entropy, within the two bounds."""
    g, H, W, dloss = inputs(90, 700, 128, BF, 5)
    y = labels_of(g, 90, 700)
    wide_ids = torch.full((90, 4), 3, device="cuda", dtype=torch.int64)
    wide_ids[:, 1] = y
    wide_t = torch.full((90, 3), float("nan"), device="cuda")
    wide_t[:, 2] = 4.0
    loss, lse, z = mo.topk_distill_forward(H, W, wide_ids[:, 1:2], wide_t[:, 2:3])
    dH, dW = mo.topk_distill_backward(H, W, wide_ids[:, 1:2], wide_t[:, 2:3], lse, z, dloss)
    torch.cuda.synchronize()
    compare((loss, lse), R.head(H, W, dloss, labels=y), dH, dW)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_rows_may_hold_anything(gpu, dtype):
    """NaN, infinities and the type's lowest value in the H rows of positions without
    a target, and of rows whose dloss is 0: no result changes."""
    g, H, W, dloss = inputs(150, 600, 96, dtype, 9)
    y = labels_of(g, 150, 600)
    clean = run_xent(H, W, y, dloss)
    dead = ((y < 0) | (y >= 600)).nonzero()[:, 0]
    bad = H.clone()
    for i, v in zip(dead.tolist(), [float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min] * 40):
        bad[i] = v
    got = run_xent(bad, W, y, dloss)
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[0][1], clean[0][1])
    assert torch.equal(got[1], clean[1]) and torch.equal(got[2], clean[2])
    # a row left out by its weight
    bad = H.clone()
    bad[1] = float("nan")
    dH, dW = mo.softmax_xent_backward(bad, W, y, clean[0][0], clean[0][1], dloss)
    torch.cuda.synchronize()
    assert torch.equal(dH, clean[1]) and torch.equal(dW, clean[2])


def test_no_row_counts(gpu):
    _, H, W, dloss = inputs(70, 300, 64, BF, 11)
    y = torch.full((70,), -1, device="cuda", dtype=torch.int64)
    (loss, lse), dH, dW = run_xent(H, W, y, dloss)
    for t in (loss, lse, dH, dW):
        assert bool((t == 0).all())


def test_extreme_logits(gpu):
    """Logits of hundreds: the exponentials neither overflow nor lose the loss; and a
    label the model is sure of has a gradient near 0."""
    g, H, W, dloss = inputs(66, 400, 64, F32, 12)
    H = H * 60
    y = torch.randint(0, 400, (66,), generator=g, device="cuda")
    y[:20] = (H @ W.t()).argmax(1)[:20]
    got, dH, dW = run_xent(H, W, y, dloss)
    compare(got, R.head(H, W, dloss, labels=y), dH, dW)


@pytest.mark.parametrize("dtype,n,vocab,dim", [(BF, 4096, 100003, 64), (F32, 2048, 40009, 40), (BF, 1, 60001, 320)])
def test_vocabulary_in_pieces(gpu, dtype, n, vocab, dim):
    """Vocabularies that take several pieces (and one that takes many tiles for one
    token), the last piece ragged."""
    g, H, W, dloss = inputs(n, vocab, dim, dtype, 21)
    y = labels_of(g, n, vocab)
    y[-1] = vocab - 1
    got, dH, dW = run_xent(H, W, y, dloss)
    # the reference in groups of rows, whose parts add up
    want_w, bound_w = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda"), 0.0
    for r in range(0, n, 512):
        s = slice(r, min(n, r + 512))
        want = R.head(H[s], W, dloss[s], labels=y[s])
        R.check(got[0][s], want["loss"], want["b_loss"], "loss")
        R.check(got[1][s], want["lse"], want["b_lse"], "lse")
        R.check(dH[s], want["dH"], want["b_dH"], "dH")
        want_w += want["dW"]
        bound_w = bound_w + want["b_dW"]
    # each group's bound counts its own terms; a sum over n rows has n / 512 times as many
    R.check(dW, want_w, bound_w * max(1, n // 512) + R.ut(dtype) * want_w.abs(), "dW")


@pytest.mark.parametrize("n", [40, 300])
def test_one_gradient_at_a_time_and_reproducible(gpu, n):
    g, H, W, dloss = inputs(n, 2100, 256, BF, 31)
    y = labels_of(g, n, 2100)
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, dW = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
    ws = torch.full((mo.softmax_xent_workspace_bytes(H, W, backward=True),), 255, dtype=torch.uint8, device="cuda")
    a, none = mo.softmax_xent_backward(H, W, y, loss, lse, dloss, need_dW=False, workspace=ws)
    assert none is None
    none, b = mo.softmax_xent_backward(H, W, y, loss, lse, dloss, need_dH=False, workspace=ws)
    assert none is None
    fw = torch.full((mo.softmax_xent_workspace_bytes(H, W),), 255, dtype=torch.uint8, device="cuda")
    loss2, lse2 = mo.softmax_xent_forward(H, W, y, workspace=fw)
    torch.cuda.synchronize()
    assert torch.equal(a, dH) and torch.equal(b, dW) and torch.equal(loss, loss2) and torch.equal(lse, lse2)


def test_empty_batch(gpu):
    W = torch.ones(300, 64, device="cuda", dtype=BF)
    H, y = torch.zeros(0, 64, device="cuda", dtype=BF), torch.zeros(0, device="cuda", dtype=torch.int64)
    loss, lse = mo.softmax_xent_forward(H, W, y)
    dH, dW = mo.softmax_xent_backward(H, W, y, loss, lse, loss)
    torch.cuda.synchronize()
    assert loss.shape == (0,) and dH.shape == (0, 64) and bool((dW == 0).all())


@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_gradient_by_differences(gpu, kind):
    """fp32 gradients against central differences of the 64-bit loss (step 1e-5: the
    truncation is below 1e-8 of the sum of magnitudes, the gradients' own error 1e-5)."""
    g, H, W, dloss = inputs(30, 200, 48, F32, 41)
    if kind == "xent":
        kw = dict(labels=labels_of(g, 30, 200))
        loss, lse = mo.softmax_xent_forward(H, W, kw["labels"])
        dH, dW = mo.softmax_xent_backward(H, W, kw["labels"], loss, lse, dloss)
    else:
        ids = torch.randint(0, 200, (30, 6), generator=g, device="cuda")
        kw = dict(ids=ids, teacher=rand(g, (30, 6), F32, 2.0), T=1.5)
        loss, lse, z = mo.topk_distill_forward(H, W, ids, kw["teacher"], temperature=1.5)
        dH, dW = mo.topk_distill_backward(H, W, ids, kw["teacher"], lse, z, dloss, temperature=1.5)
    torch.cuda.synchronize()
    f = lambda h, w: float((R.head(h, w, **kw)["loss"] * dloss.double()).sum())
    for grad, k in ((dH, 0), (dW, 1)):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        p, m = [H.double(), W.double()], [H.double(), W.double()]
        p[k], m[k] = p[k] + 1e-5 * v, m[k] - 1e-5 * v
        num = (f(*p) - f(*m)) / 2e-5
        assert abs(float((grad.double() * v).sum()) - num) <= 1e-5 * float((grad.double() * v).abs().sum()) + 1e-9


@pytest.mark.parametrize("kind", ["mean", "far apart", "infinite first", "none", "tiny first"])
def test_weights_of_the_rows(gpu, kind):
    """dloss of one value (a mean), over many orders of magnitude, with zeros and a
    non-finite weight in the first rows, and of zeros only."""
    g, H, W, _ = inputs(200, 500, 96, BF, 51)
    y = torch.randint(0, 500, (200,), generator=g, device="cuda")
    if kind == "mean":
        dloss = torch.full((200,), 1 / 200, device="cuda")
    elif kind == "far apart":
        dloss = 10.0 ** torch.linspace(-12, 6, 200, device="cuda")
    elif kind == "infinite first":
        dloss = torch.full((200,), -0.3, device="cuda")
        dloss[:70] = 0
        y[1] = -1
        dloss[1] = float("inf")          # a masked row's weight does not count either
    elif kind == "tiny first":
        dloss = torch.full((200,), 0.7, device="cuda")
        dloss[:128] = 0
        dloss[5] = 1e-30
    else:
        dloss = torch.zeros(200, device="cuda")
    got, dH, dW = run_xent(H, W, y, dloss)
    compare(got, R.head(H, W, torch.where(y < 0, torch.zeros_like(dloss), dloss), labels=y), dH, dW)


def test_a_mean_loses_no_precision(gpu):
    """With equal weights the gradients' error stays near the rounding of the results
    (uniform mantissas: 2^-8 / sqrt(12) of a value on average, 1.7e-3 with the
    spread of mantissas): delta's own rounding, independent of it and of at most
    the same size, adds at most a factor sqrt(2)."""
    g = gen(61)
    n, vocab, dim = 700, 5000, 512
    W = rand(g, (vocab, dim), BF, 0.02)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    H = (torch.randn((n, dim), generator=g, device="cuda") + 30 * W[y].float()).to(BF)
    for count in (n, 641, 911, 1021):
        dloss = torch.full((n,), 1 / count, device="cuda")
        _, dH, dW = run_xent(H, W, y, dloss)
        want = R.head(H, W, dloss, labels=y)
        for got, name in ((dH, "dH"), (dW, "dW")):
            exact = want[name]
            own = float((exact.to(BF).double() - exact).norm() / exact.norm())
            err = float((got.double() - exact).norm() / exact.norm())
            assert err <= 1.45 * own, (count, name, err, own)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 2000), (34, 700, 2000), (65, 1111, 777), (300, 520, 3000),
                                         (129, 257, 64), (20, 20000, 1024)])
def test_long_products_of_few_tiles(gpu, n, vocab, dim, dtype):
    """Few tiles with a long product: K is split over the workgroups."""
    g, H, W, dloss = inputs(n, vocab, dim, dtype, n + dim)
    y = labels_of(g, n, vocab)
    got, dH, dW = run_xent(H, W, y, dloss)
    compare(got, R.head(H, W, dloss, labels=y), dH, dW)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,dim", [(2000, 300, 100), (1787, 1000, 404), (5000, 40, 64), (900, 513, 130)])
def test_many_tokens_of_a_small_vocabulary(gpu, n, vocab, dim, dtype):
    """dW of few tiles with many tokens: its sums over the tokens are split as well."""
    g, H, W, dloss = inputs(n, vocab, dim, dtype, n + vocab)
    y = labels_of(g, n, vocab)
    got, dH, dW = run_xent(H, W, y, dloss, 3)
    compare(got, R.head(H, W, dloss, labels=y), dH, dW)
    again = mo.softmax_xent_backward(H, W, y, *got, dloss)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)


def test_split_products_in_two_pieces(gpu):
    """The longest rows there are: two pieces of the vocabulary, each split along K."""
    g, H, W, dloss = inputs(5, 2000, 65536, F32, 71)
    y = labels_of(g, 5, 2000)
    got, dH, dW = run_xent(H, W, y, dloss)
    compare(got, R.head(H, W, dloss, labels=y), dH, dW)


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 4), (5, 300, 20), (64, 513, 36), (130, 256, 100), (63, 1000, 1028),
                                         (3, 20000, 8), (512, 700, 260), (513, 300, 128)])
def test_fp32_head_read_in_place(gpu, n, vocab, dim, pad):
    """Rows of whole 16 bytes: up to 512 tokens W is read as it lies, with ends of dim
    and of the vocabulary inside a tile and a stage; 513 tokens take the copies."""
    g, H, W, dloss = inputs(n, vocab, dim, F32, n + vocab + dim, pad)
    y = labels_of(g, n, vocab)
    got, dH, dW = run_xent(H, W, y, dloss, pad)
    compare(got, R.head(H, W, dloss, labels=y), dH, dW)


def test_fp32_values_of_the_whole_range(gpu):
    """Values that would round to infinity in bf16, and ones with few significant bits."""
    g, H, W, dloss = inputs(40, 300, 64, F32, 83)
    y = labels_of(g, 40, 300)
    W[7] = torch.finfo(F32).max                      # finite, beyond the largest bf16
    H *= 1e-30
    W[8] = 2.0 ** torch.arange(64, device="cuda")
    got, dH, dW = run_xent(H, W, y, dloss)
    assert torch.isfinite(dH).all() and torch.isfinite(dW).all()
    want = R.head(H, W, dloss, labels=y)
    for k, v in (("loss", got[0]), ("lse", got[1])):
        assert ((v.double() - want[k]).abs() <= want["b_" + k]).all()


@pytest.mark.parametrize("n", [40, 600])
def test_fp32_infinities_stay_visible(gpu, n):
    """An infinity or NaN in a row of W reaches every token's loss as a value that is
    not finite; one in a masked token's H reaches nothing."""
    g, H, W, dloss = inputs(n, 300, 64, F32, 89)
    y = torch.randint(0, 300, (n,), generator=g, device="cuda")
    y[5] = -1
    H[5] = float("inf")
    got, dH, dW = run_xent(H, W, y, dloss)
    clean = H.clone()
    clean[5] = 0
    base, bH, bW = run_xent(clean, W, y, dloss)
    assert all(torch.equal(a, b) for a, b in zip((*got, dH, dW), (*base, bH, bW)))
    for bad in (float("inf"), float("nan")):
        V = W.clone()
        V[9, 3] = bad
        loss, lse = mo.softmax_xent_forward(clean, V, y)
        live = y >= 0
        # 0 x infinity or a positive infinity; a logit of minus infinity is a finite loss
        assert (~torch.isfinite(lse[live])).any() and loss[5] == 0 and lse[5] == 0


@pytest.mark.parametrize("n,vocab,dim,k", [(3, 5000, 64, 0), (70, 3000, 513, 0), (2, 4000, 72, 5), (70, 3000, 96, 9),
                                           (600, 2000, 260, 17)])
def test_targets_lose_no_precision_in_dH(gpu, n, vocab, dim, k):
    """Logits near zero: delta is about 1 / vocab away from the targets, so what its
    rounding there adds to dH is at most 2^-8 / sqrt(vocab / targets) of it, and the
    targets' own rounding is made up for: dH is as near as its rounding to bf16
    (2 % more for the rest: 2^-8 / sqrt(2000 / 17) against 1.7e-3, in squares)."""
    g = gen(97 + n)
    W = rand(g, (vocab, dim), BF, 1.0)
    H = rand(g, (n, dim), BF, 1e-3)
    dloss = torch.rand(n, generator=g, device="cuda") + 0.1
    if k:
        ids = torch.randint(0, vocab, (n, k), generator=g, device="cuda")
        ids[:, -1] = ids[:, 0]                       # one id twice
        ids[0, 1] = -1
        t = torch.randn((n, k), generator=g, device="cuda")
        _, lse, z = mo.topk_distill_forward(H, W, ids, t)
        dH, _ = mo.topk_distill_backward(H, W, ids, t, lse, z, dloss)
        want = R.head(H, W, dloss, ids=ids, teacher=t)["dH"]
    else:
        y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
        loss, lse = mo.softmax_xent_forward(H, W, y)
        dH, _ = mo.softmax_xent_backward(H, W, y, loss, lse, dloss)
        want = R.head(H, W, dloss, labels=y)["dH"]
    own = float((want.to(BF).double() - want).norm())
    err = float((dH.double() - want).norm())
    assert err <= 1.02 * own, err / own
