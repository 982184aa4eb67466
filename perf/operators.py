"""The model-end operators as a training or evaluation program calls them: the
embedding lookup and its gradient, the layer norm and its gradients, the
softmax cross entropy of the output head, and distillation from a teacher's top
logits.  ``own`` false computes each in elementary torch operations, ``own``
true through ``matrix_optimizers_amd``.

Shapes: the 128256 x 4096 output head and the 8192-wide matrices of the large
Muon bucket, the hidden sizes 2048 and 4096 of the decoder-layer buckets, and
odd sizes around them.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}
DEV = "cuda"
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # embedding rows of the eight sequences of a small decoding batch
        {"name": "embed_fwd_8", "op": "embed_fwd", "tokens": 8, "vocab": 128256, "dim": 4096,
         "type": BF16, "pad": False},
        # the same lookup for a training micro-batch of eight 2048-token sequences
        {"name": "embed_fwd_16384", "op": "embed_fwd", "tokens": 16384, "vocab": 128256, "dim": 4096,
         "type": BF16, "pad": False},
        # the gradient of that micro-batch's embedding, the whole matrix written
        {"name": "embed_bwd_16384", "op": "embed_bwd", "tokens": 16384, "vocab": 128256, "dim": 4096,
         "type": BF16, "pad": False},
        # a short, padded, odd-sized batch on an fp32 model
        {"name": "embed_bwd_1023_f32", "op": "embed_bwd", "tokens": 1023, "vocab": 32001, "dim": 2048,
         "type": F32, "pad": True},
        # one norm in a decoding step of eight sequences
        {"name": "norm_fwd_8_f32", "op": "norm_fwd", "rows": 8, "dim": 2048, "type": F32},
        # one norm over a training micro-batch of a hidden-8192 model
        {"name": "norm_fwd_16384", "op": "norm_fwd", "rows": 16384, "dim": 8192, "type": BF16},
        # one norm's gradients over an odd number of tokens (packed sequences)
        {"name": "norm_bwd_16381", "op": "norm_bwd", "rows": 16381, "dim": 4096, "type": BF16},
        # the loss and its gradients for one sequence of 8192 tokens on the full head
        {"name": "xent_step_8192", "op": "xent_step", "tokens": 8192, "vocab": 128256, "dim": 4096,
         "type": BF16, "pad": True},
        # scoring a handful of continuations: the loss alone, few tokens
        {"name": "xent_fwd_37", "op": "xent_fwd", "tokens": 37, "vocab": 128256, "dim": 4096,
         "type": BF16, "pad": False},
        # an fp32 model with a small vocabulary, odd sizes, padded batch
        {"name": "xent_step_1021_f32", "op": "xent_step", "tokens": 1021, "vocab": 32001, "dim": 1000,
         "type": F32, "pad": True},
        # a student's step against a teacher's 64 stored logits per token
        {"name": "distill_step_4096", "op": "distill_step", "tokens": 4096, "vocab": 128256, "dim": 2048,
         "top": 64, "temperature": 2.0, "type": BF16, "pad": False},
        # a short distillation batch with few stored logits, some rows without any
        {"name": "distill_step_257", "op": "distill_step", "tokens": 257, "vocab": 32001, "dim": 2048,
         "top": 10, "temperature": 1.0, "type": BF16, "pad": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """A row length: a multiple of 64 two times in three, any length otherwise."""
    d = _log(rng, lo, hi)
    return max(lo, d // 64 * 64) if rng.random() < 2 / 3 else d


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "xent_fwd", "xent_step",
                     "distill_step"])
    ty = rng.choice([BF16, BF16, F32])
    if op.startswith("norm"):
        rows, dim = _log(rng, 1, 32768), _width(rng, 64, 16384)
        return {"op": op, "rows": min(rows, (1 << 28) // dim), "dim": dim, "type": ty}
    vocab = _log(rng, 1000, 131072)
    if op.startswith("embed"):
        return {"op": op, "tokens": _log(rng, 1, 32768), "vocab": vocab, "dim": _width(rng, 64, 8192),
                "type": ty, "pad": rng.random() < 0.5}
    dim = _width(rng, 64, 8192)
    # at most a quarter of the largest listed step's products
    tokens = min(_log(rng, 1, 8192), max(1, (8192 * 128256 * 1024) // (vocab * dim)))
    case = {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "type": ty, "pad": rng.random() < 0.5}
    if op == "distill_step":
        case["top"] = _log(rng, 1, 256)
        case["temperature"] = rng.choice([1.0, 1.5, 2.0, 4.0])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _zipf(g, n, vocab):
    """Ids with frequency about 1 / (id + 1), as the tokens of a text."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)


def _randn(g, shape, std, ty):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(DT[ty])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, ty, dim = case["op"], case["type"], case["dim"]
    st = {"op": op}
    if op.startswith("norm"):
        rows = case["rows"]
        # rows of a residual stream: their own scale and mean
        x = torch.randn((rows, dim), generator=g, device=DEV)
        x *= 0.5 + 2 * torch.rand((rows, 1), generator=g, device=DEV)
        x += 0.2 * torch.randn((rows, 1), generator=g, device=DEV)
        st["x"] = x.to(DT[ty])
        # weight and bias are slices of the packed fp32 tail
        st["w"] = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
        st["b"] = 0.1 * torch.randn(dim, generator=g, device=DEV)
        if op == "norm_bwd":
            st["dy"] = _randn(g, (rows, dim), 1e-2, ty)
            xd = st["x"].double()
            mean = xd.mean(1)
            var = (xd - mean[:, None]).pow_(2).mean(1)
            # what the forward pass left for the backward
            st["mean"] = mean.float()
            st["rstd"] = (var + EPS).rsqrt().float()
        return st
    n, vocab = case["tokens"], case["vocab"]
    ids = _zipf(g, n, vocab)
    if case["pad"]:   # one position in sixteen is padding
        ids[torch.rand(n, generator=g, device=DEV) < 1 / 16] = -100
    if op == "embed_fwd":
        st["tokens"], st["scale"] = ids, math.sqrt(dim)
        st["W"] = _randn(g, (vocab, dim), 0.02, ty)
        return st
    if op == "embed_bwd":
        st["tokens"], st["scale"] = ids, math.sqrt(dim)
        st["dY"] = _randn(g, (n, dim), 1e-3, ty)
        st["G"] = torch.empty((vocab, dim), device=DEV, dtype=DT[ty])   # the optimizer's gradient
        return st
    W = _randn(g, (vocab, dim), 0.02, ty)
    H = torch.randn((n, dim), generator=g, device=DEV)
    # a model that has learnt something: the label's logit stands out by about 6
    H += (6 / (dim * 4e-4)) * W[ids.clamp(min=0)].float()
    st["H"], st["W"] = H.to(DT[ty]), W
    if op == "distill_step":
        k = case["top"]
        top = (ids.clamp(min=0)[:, None] + torch.arange(k, device=DEV) * max(1, vocab // k)) % vocab
        gap = torch.rand((n, k), generator=g, device=DEV)
        st["teacher"] = 12 - torch.cumsum(gap, 1) * (8 / k + 0.05)
        if case["pad"]:
            # a teacher that stored fewer logits for some tokens, none for the padding
            cut = torch.rand((n, 1), generator=g, device=DEV) * 4 * k
            top[torch.arange(k, device=DEV) >= cut] = -1
            top[ids < 0] = -1
        st["ids"], st["T"] = top, case["temperature"]
        valid = (top >= 0).any(1)
    else:
        st["labels"] = ids
        valid = ids >= 0
    if op != "xent_fwd":
        # the mean over the rows that count
        st["dloss"] = valid.float() / valid.sum().clamp(min=1)
        st["dW"] = torch.empty_like(W)   # the optimizer's gradient
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _head_grads(p, coef, H, W, Hf, Wf):
    """dH and dW from the logits' gradients p (per row still without coef)."""
    d = torch.where((coef != 0)[:, None], p * coef[:, None], torch.zeros_like(p))
    return (d @ Wf).to(H.dtype), (d.t() @ Hf).to(W.dtype)


def _plain(st):
    op = st["op"]
    if op == "norm_fwd":
        x = st["x"].float()
        mean = x.mean(1, keepdim=True)
        c = x - mean
        rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        return (c * rstd * st["w"] + st["b"]).to(st["x"].dtype), mean[:, 0], rstd[:, 0]
    if op == "norm_bwd":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = (st["x"].float() - st["mean"][:, None]) * rstd
        gw = dy * st["w"]
        dx = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
        return dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    if op == "embed_fwd":
        t, W = st["tokens"], st["W"]
        ok = t >= 0
        y = W[t.clamp(min=0)].float() * st["scale"]
        return torch.where(ok[:, None], y, torch.zeros_like(y)).to(W.dtype)
    if op == "embed_bwd":
        t, dY, G = st["tokens"], st["dY"], st["G"]
        ok = t >= 0
        acc = torch.zeros(G.shape, device=G.device, dtype=torch.float32)
        acc.index_add_(0, t[ok], dY[ok].float())
        return (acc * st["scale"]).to(G.dtype)
    H, W = st["H"], st["W"]
    Hf, Wf = H.float(), W.float()
    z = Hf @ Wf.t()
    if op == "distill_step":
        ids, T = st["ids"], st["T"]
        on = ids >= 0
        has = on.any(1)
        at = ids.clamp(min=0)
        t = torch.where(on, st["teacher"].float() / T, torch.full_like(st["teacher"], -math.inf))
        t = torch.where(has[:, None], t, torch.zeros_like(t))
        et = torch.exp(t - t.amax(1, keepdim=True))
        st_ = et.sum(1, keepdim=True)
        pt = torch.where(on, et / st_, torch.zeros_like(et))
        logpt = t - t.amax(1, keepdim=True) - torch.log(st_)
        ztop = torch.gather(z, 1, at)
        z = z / T
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        s = e.sum(1, keepdim=True)
        lse = m + torch.log(s)
        kl = torch.where(pt > 0, pt * (logpt - (ztop / T - lse)), torch.zeros_like(pt)).sum(1)
        loss = torch.where(has, T * T * kl, torch.zeros_like(kl))
        q = e / s
        q.scatter_add_(1, at, -pt)
        dH, dW = _head_grads(q, torch.where(has, st["dloss"] * T, torch.zeros_like(kl)), H, W, Hf, Wf)
        return loss, dH, dW
    y = st["labels"]
    ok = y >= 0
    zy = torch.gather(z, 1, y.clamp(min=0)[:, None])
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    loss = (m + torch.log(s) - zy)[:, 0]
    loss = torch.where(ok, loss, torch.zeros_like(loss))
    if op == "xent_fwd":
        lse = (m + torch.log(s))[:, 0]
        return loss, torch.where(ok, lse, torch.zeros_like(lse))
    p = e / s
    p.scatter_add_(1, y.clamp(min=0)[:, None], -torch.ones_like(zy))
    dH, dW = _head_grads(p, torch.where(ok, st["dloss"], torch.zeros_like(loss)), H, W, Hf, Wf)
    return loss, dH, dW


def _own(st):
    import matrix_optimizers_amd as mo
    op = st["op"]
    if op == "norm_fwd":
        return mo.layer_norm_forward(st["x"], st["w"], st["b"], eps=EPS)
    if op == "norm_bwd":
        return mo.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["w"])
    if op == "embed_fwd":
        return mo.embedding_forward(st["tokens"], st["W"], scale=st["scale"])
    if op == "embed_bwd":
        return mo.embedding_backward(st["tokens"], st["dY"], st["G"], scale=st["scale"])
    H, W = st["H"], st["W"]
    if op == "distill_step":
        ids, teacher, T = st["ids"], st["teacher"], st["T"]
        loss, lse, z = mo.topk_distill_forward(H, W, ids, teacher, temperature=T)
        dH, dW = mo.topk_distill_backward(H, W, ids, teacher, lse, z, st["dloss"], temperature=T,
                                          dW=st["dW"])
        return loss, dH, dW
    loss, lse = mo.softmax_xent_forward(H, W, st["labels"])
    if op == "xent_fwd":
        return loss, lse
    dH, dW = mo.softmax_xent_backward(H, W, st["labels"], loss, lse, st["dloss"], dW=st["dW"])
    return loss, dH, dW


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the least a pass has to move and compute
# ---------------------------------------------------------------------------

def work(case):
    op, dim = case["op"], case["dim"]
    es = 2 if case["type"] == BF16 else 4
    if op.startswith("norm"):
        n = case["rows"] * dim
        if op == "norm_fwd":
            return {"bytes": 2 * n * es + 8 * dim + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * es + 12 * dim + 8 * case["rows"], "flops": 14 * n}
    n, vocab = case["tokens"], case["vocab"]
    if op == "embed_fwd":
        # at most `vocab` distinct rows are read
        return {"bytes": (min(n, vocab) + n) * dim * es + 8 * n, "flops": n * dim}
    if op == "embed_bwd":
        return {"bytes": (n + vocab) * dim * es + 8 * n, "flops": n * dim + vocab * dim}
    k = case.get("top", 1)
    head = (n + vocab) * dim * es + n * k * (12 if op == "distill_step" else 8)
    if op == "xent_fwd":
        return {"bytes": head + 8 * n, "flops": 2 * n * vocab * dim}
    # logits, dH = d W, dW = d^T H
    return {"bytes": 2 * (n + vocab) * dim * es + n * k * (12 if op == "distill_step" else 8) + 8 * n,
            "flops": 6 * n * vocab * dim}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(st, op)
    if op == "embed_fwd":
        W, t = st["W"], st["tokens"].tolist()
        out = torch.zeros((len(t), W.shape[1]), device=DEV, dtype=torch.float64)
        keep = [i for i, v in enumerate(t) if v >= 0]
        out[keep] = W[[t[i] for i in keep]].double()
        return out.mul_(st["scale"])
    if op == "embed_bwd":
        # row v: the sum of its tokens' rows, by differences of running sums over the sorted tokens
        t, dY, G = st["tokens"], st["dY"], st["G"]
        order = torch.argsort(t, stable=True)
        edge = torch.searchsorted(t[order], torch.arange(G.shape[0] + 1, device=DEV))
        out = torch.empty(G.shape, device=DEV, dtype=torch.float64)
        for c in range(0, G.shape[1], 256):
            run_ = torch.zeros((len(t) + 1, min(256, G.shape[1] - c)), device=DEV, dtype=torch.float64)
            torch.cumsum(dY[order, c:c + 256].double(), 0, out=run_[1:])
            out[:, c:c + 256] = (run_[edge[1:]] - run_[edge[:-1]]) * st["scale"]
        absent = edge[1:] == edge[:-1]
        out[absent] = 0
        return out
    return _exact_head(st, op)


def _exact_norm(st, op):
    step = max(1, (1 << 26) // st["x"].shape[1])
    w, b = st["w"].double(), st["b"].double()
    if op == "norm_fwd":
        parts = []
        for x in st["x"].split(step):
            x = x.double()
            var, mean = torch.var_mean(x, 1, correction=0)
            inv = (var + EPS) ** -0.5
            parts.append(((x - mean[:, None]) * inv[:, None] * w + b, mean, inv))
        return tuple(torch.cat(p) for p in zip(*parts))
    dim = st["x"].shape[1]
    dxs, dw, db = [], torch.zeros_like(w), torch.zeros_like(w)
    for x, dy, mean, inv in zip(st["x"].split(step), st["dy"].split(step), st["mean"].split(step),
                                st["rstd"].split(step)):
        x, dy, inv = x.double(), dy.double(), inv.double()[:, None]
        n = (x - mean.double()[:, None]) * inv
        up = dy * w
        proj = (up * n).sum(1, keepdim=True) / dim
        dxs.append(inv * (up - up.sum(1, keepdim=True) / dim - n * proj))
        dw += (dy * n).sum(0)
        db += dy.sum(0)
    return torch.cat(dxs), dw, db


def _exact_head(st, op):
    """Rows in groups: logits, log-softmax, the targets' distribution subtracted."""
    H, W = st["H"], st["W"].double()
    n, (vocab, dim) = H.shape[0], W.shape
    group = max(1, (1 << 28) // vocab)
    losses, lses, dHs = [], [], []
    dW = torch.zeros((vocab, dim), device=DEV, dtype=torch.float64) if op != "xent_fwd" else None
    for r in range(0, n, group):
        rows = slice(r, min(n, r + group))
        h = H[rows].double()
        T = st["T"] if op == "distill_step" else 1.0
        z = torch.mm(h, W.t()) / T
        logq = torch.log_softmax(z, 1)
        lse = z[:, 0] - logq[:, 0]
        del z
        if op == "distill_step":
            ids, t = st["ids"][rows], st["teacher"][rows].double() / T
            gone = ids < 0
            live = ~gone.all(1)
            t = t.masked_fill(gone, -math.inf).masked_fill(~live[:, None], 0.0)
            logp = torch.log_softmax(t, 1)
            p = logp.exp().masked_fill(gone, 0.0)
            lq = logq.gather(1, ids.clamp(min=0))
            loss = T * T * torch.where(p > 0, p * (logp - lq), 0.0).sum(1)
        else:
            ids = st["labels"][rows, None]
            live = ids[:, 0] >= 0
            p = (ids >= 0).double()
            loss = -logq.gather(1, ids.clamp(min=0))[:, 0]
        losses.append(loss.masked_fill(~live, 0.0))
        lses.append(lse.masked_fill(~live, 0.0))
        if dW is None:
            continue
        c = (st["dloss"][rows].double() * T).masked_fill(~live, 0.0)[:, None]
        d = logq.exp_().mul_(c)
        d.scatter_add_(1, ids.clamp(min=0), -(p * c))
        dHs.append(torch.mm(d, W))
        dW.addmm_(d.t(), h)
        del d, logq
    loss = torch.cat(losses)
    return (loss, torch.cat(lses)) if dW is None else (loss, torch.cat(dHs), dW)
