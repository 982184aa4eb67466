"""Plain 64-bit forms of the embedding, layer norm, cross entropy and distillation
operators (torch float64 on any device), written from their formulas, with
element-wise bounds on how far a kernel that sums in fp32 and rounds once to the
result's type may be from them.

Bounds.  u = 2^-24 is the fp32 half unit, ut = finfo(t).eps / 2 that of the result's
type.  A sum of m terms in fp32, in any order, is off by at most m u sum|terms| to
first order; sums on the matrix cores are given 2 u per addition, since their
rounding mode is not assumed.  Second-order terms are covered by SLACK.
"""
import math

import torch

U = 2.0 ** -24
SLACK = 1.02          # second-order terms: every first-order bound here is below 1e-2
TINY = 2.0 ** -120    # subnormal inputs and results may be flushed


def ut(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, want, bound, what):
    """|got - want| <= bound element by element; prints the closest approach."""
    got, want, bound = got.double(), want.double(), bound.double() * SLACK + TINY
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    err = (got - want).abs()
    ratio = float((err / bound).max()) if err.numel() else 0.0
    assert ratio <= 1.0, f"{what}: error {ratio:.3g} of its bound (largest error {float(err.max()):.3g})"
    return ratio


# ---- embedding ---------------------------------------------------------------------

def embed(tokens, W, scale):
    ok = (tokens >= 0) & (tokens < W.shape[0])
    Y = W.double()[tokens.clamp(0, W.shape[0] - 1)] * scale
    return torch.where(ok[:, None], Y, torch.zeros_like(Y))


def embed_grad(tokens, dY, vocab, scale):
    """G and the bound of one without its own rounding: per row and column
    (terms + 2) u scale sum|dY| (the additions, the scaling, one spare)."""
    ok = (tokens >= 0) & (tokens < vocab)
    t, d = tokens[ok], dY[ok].double()
    G = torch.zeros((vocab, dY.shape[1]), dtype=torch.float64, device=dY.device)
    A = torch.zeros_like(G)
    cnt = torch.zeros(vocab, dtype=torch.float64, device=dY.device)
    G.index_add_(0, t, d)
    A.index_add_(0, t, d.abs())
    cnt.index_add_(0, t, torch.ones_like(t, dtype=torch.float64))
    return G * scale, (cnt + 2)[:, None] * U * A * abs(scale)


# ---- layer norm --------------------------------------------------------------------

def norm(X, w, b, eps):
    x = X.double()
    mu = x.mean(1)
    c = x - mu[:, None]
    r = ((c * c).mean(1) + eps) ** -0.5
    y = c * r[:, None]
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mu, r


def norm_depth(cols):
    """Additions on the longest path of a row's sum: a thread's own elements, the
    wavefront's butterfly and the waves of the workgroup."""
    return 8 * max(4, -(-cols // 8192)) + 6 + 16 + 1


def norm_bounds(X, w, b, eps, out_dtype):
    """Bounds of y, mu and r: d_mu = (D + 1) u mean|x|; the variance is off by
    2 d_mu mean|c| + (D + 4) u var, r by half of that relative to var + eps plus
    4 u; y by |w| r d_mu + |w c r| (rel r + 4 u) + u (|w c r| + |b|) + rounding."""
    y, mu, r = norm(X, w, b, eps)
    x = X.double()
    c = x - mu[:, None]
    D = norm_depth(X.shape[1])
    dmu = (D + 1) * U * x.abs().mean(1)
    var = (c * c).mean(1)
    dvar = 2 * dmu * c.abs().mean(1) + dmu * dmu + (D + 4) * U * var
    rel = 0.5 * dvar / (var + eps) + 4 * U
    aw = w.double().abs() if w is not None else torch.ones_like(x[0])
    n = aw * c.abs() * r[:, None]
    by = aw * (r * dmu)[:, None] + n * (rel[:, None] + 4 * U) + U * (n + (b.double().abs() if b is not None else 0))
    return by + ut(out_dtype) * y.abs(), dmu + U * mu.abs(), r * rel


def norm_grad(dY, X, mean, rstd, w):
    """dx, dw, db and bounds, from the fp32 mean and rstd as given."""
    x, dy, r = X.double(), dY.double(), rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * r
    g = dy * w.double() if w is not None else dy
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    D, N = norm_depth(X.shape[1]), X.shape[0]
    bx = r.abs() * ((D + 2) * U * g.abs().mean(1, keepdim=True) + (D + 6) * U * xh.abs() * (g * xh).abs().mean(1, keepdim=True)
                    + 6 * U * (g.abs() + m1.abs() + xh.abs() * m2.abs()))
    bx = bx + ut(X.dtype) * dx.abs()
    return (dx, (dy * xh).sum(0), dy.sum(0)), (bx, (N + 4) * U * (dy * xh).abs().sum(0), (N + 1) * U * dy.abs().sum(0))


# ---- output head -------------------------------------------------------------------

def targets(vocab, labels=None, ids=None, teacher=None, T=1.0):
    """(live rows, ids, p, log p): the target distribution at the ids."""
    if labels is not None:
        live = (labels >= 0) & (labels < vocab)
        p = live.double()[:, None]
        return live, labels.clamp(0, vocab - 1)[:, None], p, torch.zeros_like(p)
    on = (ids >= 0) & (ids < vocab)
    t = torch.where(on, teacher.double() / T, torch.full(ids.shape, -math.inf, dtype=torch.float64, device=ids.device))
    live = (t > -math.inf).any(1)
    t = torch.where(live[:, None], t, torch.zeros_like(t))
    logp = torch.log_softmax(t, 1)
    p = torch.where(on & live[:, None], logp.exp(), torch.zeros_like(t))
    return live, ids.clamp(0, vocab - 1), p, torch.where(p > 0, logp, torch.zeros_like(logp))


def head(H, W, dloss=None, labels=None, ids=None, teacher=None, T=1.0):
    """loss, lse, the gradients for dloss, and bounds of all four."""
    h, w = H.double(), W.double()
    N, (V, d) = H.shape[0], W.shape
    live, at, p, logp = targets(V, labels, ids, teacher, T)
    h = torch.where(live[:, None], h, torch.zeros_like(h))   # masked rows may hold anything
    f32 = H.dtype == torch.float32
    z = h @ w.t()
    # the product's sum (six times as many terms for fp32) and its dropped parts
    az = h.abs() @ w.abs().t()
    dz = 2 * U * d * (6 if f32 else 1) * az + (2.0 ** -22 * az if f32 else 0)
    dzt = torch.gather((d + 8) * U * az, 1, at)              # the gathered dot products
    z, dz = z / T, dz / T + 4 * U * z.abs() / T
    lse = torch.logsumexp(z, 1)
    q = (z - lse[:, None]).exp()
    # exponentials within 2^-21, log2 / natural conversions within 4 u of their
    # arguments, sums of V positive terms along at most 160 + V / 8192 additions
    dlse = (q * dz).sum(1) + 2.0 ** -21 + (160 + V / 8192) * U + 6 * U * (lse.abs() + z.abs().amax(1))
    zt = torch.gather(z, 1, at)
    if labels is not None:
        loss = torch.where(live, lse - zt[:, 0], torch.zeros_like(lse))
        dl = dlse + dzt[:, 0] + U * loss.abs()
    else:
        k = at.shape[1]
        terms = torch.where(p > 0, p * (logp - (zt - lse[:, None])), torch.zeros_like(p))
        loss = T * T * terms.sum(1)
        # p within (k + 40) u + 4 u |t| of itself: |t / T - max| <= |logp| + log k
        dp = (k + 40 + 8 * (logp.abs() + math.log(k + 1))) * U
        dlogp = dp
        loss_abs = p * (logp.abs() + zt.abs() + lse.abs()[:, None])
        dl = T * T * ((dp + (k + 8) * U) * loss_abs + p * (dlogp + dzt / T + 2 * U * zt.abs() + dlse[:, None])).sum(1)
    loss = torch.where(live, loss, torch.zeros_like(loss))
    lse_out = torch.where(live, lse, torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse_out, "b_loss": dl, "b_lse": dlse + U * lse.abs(), "live": live}
    if dloss is None:
        return out
    c = torch.where(live, dloss.double() * T, torch.zeros_like(loss))[:, None]
    delta = q.clone()
    delta.scatter_add_(1, at, -p)
    delta = c * delta
    rel = dz + dlse[:, None] + 2.0 ** -21 + 6 * U * (z.abs() + lse.abs()[:, None])
    bd = c.abs() * q * rel + ut(H.dtype) * delta.abs()
    if labels is not None:
        # expm1 of the loss as stored
        extra = c[:, 0].abs() * ((-loss).exp() * dl + 8 * U)
        bd.scatter_add_(1, at, (extra * live)[:, None])
    else:
        extra = c.abs() * ((dp + 8 * U) * p + torch.gather(q, 1, at) * (dzt / T + 8 * U * zt.abs()))
        bd.scatter_add_(1, at, extra * (p > 0))
    six = 6 if f32 else 1
    drop = 2.0 ** -22 if f32 else 0.0
    # the sums times the common scale of dloss: one product more (delta's division by
    # it is within the 2^-21 above)
    out["dH"] = delta @ w
    out["b_dH"] = (bd + (2 * U * six * V + drop) * delta.abs()) @ w.abs() + (ut(H.dtype) + U) * out["dH"].abs()
    out["dW"] = delta.t() @ h
    out["b_dW"] = (bd + (2 * U * six * N + drop) * delta.abs()).t() @ h.abs() + (ut(H.dtype) + U) * out["dW"].abs()
    return out
