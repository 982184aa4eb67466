"""The operators of a layer that multiplies in 8 bits, as a training or evaluation
program calls them: the root-mean-square norm with the residual's addition (its
result in the model's type or in 8 bits) and its gradients, activations and weights
in 8 bits with a power-of-two scale for each block of 128, the product of two such
matrices, and the weight's gradient from an activation kept in 8 bits.  ``own`` false
computes each in elementary torch operations, ``own`` true through
``matrix_optimizers_amd``.

A block of 128 elements (of a row; 128 x 128 for a weight) is held as e4m3 numbers q
and a scale 2^e (one e8m0 byte), x = q 2^e, with e the least exponent for which no
element of the block is over e4m3's largest, 448; e is -127 or more.

Shapes: the 4096 x 4096, 4096 x 14336 and 8192-wide matrices of the Muon buckets, the
hidden sizes 2048 and 4096 of the decoder-layer buckets, and odd sizes around them.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}
Q8, S8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DEV = "cuda"
EPS = 1e-6
B = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one norm in a decoding step of eight sequences, its result for an 8-bit product
        {"name": "norm8_8", "op": "norm8", "rows": 8, "dim": 4096, "type": BF16, "residual": True},
        # the same over a training micro-batch of a hidden-8192 model
        {"name": "norm8_16384", "op": "norm8", "rows": 16384, "dim": 8192, "type": BF16, "residual": True},
        # an fp32 model of odd sizes
        {"name": "norm_1021_f32", "op": "norm", "rows": 1021, "dim": 1000, "type": F32, "residual": True},
        # the norm's gradients over an odd number of tokens (packed sequences)
        {"name": "norm_bwd_16381", "op": "norm_bwd", "rows": 16381, "dim": 4096, "type": BF16,
         "residual": True},
        # an activation of the feed-forward part kept for the backward pass
        {"name": "save_16384", "op": "quantize", "rows": 16384, "dim": 14336, "type": BF16, "pad": False},
        # a kept activation of a padded batch read back for layers that autograd runs
        {"name": "restore_16381", "op": "dequantize", "rows": 16381, "dim": 4096, "type": BF16, "pad": True},
        # a weight after an optimizer step, for the forward and the backward products
        {"name": "weight_14336", "op": "weight", "rows": 14336, "dim": 4096, "type": BF16},
        # the feed-forward product of a training micro-batch
        {"name": "matmul_16384", "op": "matmul", "tokens": 16384, "rows": 14336, "dim": 4096, "type": BF16},
        # the same weight in a decoding step of eight sequences
        {"name": "matmul_8", "op": "matmul", "tokens": 8, "rows": 14336, "dim": 4096, "type": BF16},
        # odd sizes, the result in fp32
        {"name": "matmul_1021_f32", "op": "matmul", "tokens": 1021, "rows": 2001, "dim": 1000, "type": F32},
        # that micro-batch's weight gradient, into what the Muon step reads
        {"name": "wgrad_16384", "op": "wgrad", "tokens": 16384, "rows": 14336, "dim": 4096, "type": BF16},
        # a short batch of an fp32 model of odd sizes
        {"name": "wgrad_257_f32", "op": "wgrad", "tokens": 257, "rows": 1000, "dim": 2001, "type": F32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """A row length: a multiple of 128 two times in three, any length otherwise."""
    d = _log(rng, lo, hi)
    return max(lo, d // B * B) if rng.random() < 2 / 3 else d


MOST = 16384 * 14336 * 4096


def draw(rng):
    op = rng.choice(["norm8", "norm", "norm_bwd", "quantize", "dequantize", "weight", "matmul", "matmul", "wgrad",
                     "wgrad"])
    ty = rng.choice([BF16, BF16, F32])
    if op.startswith("norm"):
        rows, dim = _log(rng, 1, 32768), _width(rng, 64, 16384)
        return {"op": op, "rows": min(rows, (1 << 27) // dim), "dim": dim, "type": ty,
                "residual": rng.random() < 2 / 3}
    if op in ("quantize", "dequantize", "weight"):
        rows, dim = _log(rng, 1, 32768), _width(rng, 1, 28672)
        case = {"op": op, "rows": min(rows, (1 << 27) // dim), "dim": dim, "type": ty}
        if op != "weight":
            case["pad"] = rng.random() < 0.5
        return case
    rows, dim = _width(rng, 16, 16384), _width(rng, 16, 16384)
    tokens = min(_log(rng, 1, 16384), max(1, MOST // (rows * dim)))
    return {"op": op, "tokens": tokens, "rows": rows, "dim": dim, "type": ty}


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------

def _blocks(v):
    """v (.., cols) as (.., blocks, 128), zeros behind the end."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % B)).unflatten(-1, (-1, B))


def _scale_of(amax):
    """The least e >= -127 with amax <= 448 2^e, as 2^e: amax = m 2^p with m in [1/2, 1)."""
    m, p = torch.frexp(amax)
    e = torch.where(m <= 0.875, p - 9, p - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    return torch.ldexp(torch.ones_like(amax), e)


def _to8(x):
    """x (rows, cols) fp32 in blocks of 128 along the rows."""
    b = _blocks(x)
    s = _scale_of(b.abs().amax(-1))
    q = (b / s[..., None]).flatten(-2)[:, :x.shape[1]]
    return q.to(Q8), s.to(S8)


def _square8(x):
    """x fp32 in blocks of 128 x 128."""
    a = _blocks(x).abs().amax(-1)
    s = _scale_of(_blocks(a.t()).amax(-1).t())
    q = x / s.repeat_interleave(B, 0)[:x.shape[0]].repeat_interleave(B, 1)[:, :x.shape[1]]
    return q.to(Q8), s.to(S8)


def _from8(q, s, rows=1):
    """The fp32 values of q under the scales s of blocks of rows x 128."""
    f = s.float()
    if rows > 1:
        f = f.repeat_interleave(rows, 0)[:q.shape[0]]
    return q.float() * f.repeat_interleave(B, 1)[:, :q.shape[1]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(g, shape, std, ty):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(DT[ty])


def _activation(g, rows, cols):
    """Rows of their own size, and one channel in 200 that stands out."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(torch.randn((rows, 1), generator=g, device=DEV) * 0.5)
    x *= torch.where(torch.rand(cols, generator=g, device=DEV) < 1 / 200, 20.0, 1.0)
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, ty, rows, dim = case["op"], case["type"], case["rows"], case["dim"]
    st = {"op": op, "type": DT[ty]}
    if op.startswith("norm"):
        st["x"] = _activation(g, rows, dim).to(DT[ty])
        # the weight is a slice of the packed fp32 tail
        st["w"] = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
        st["residual"] = _randn(g, (rows, dim), 2.0, ty) if case["residual"] else None
        if op == "norm_bwd":
            st["dy"] = _randn(g, (rows, dim), 1e-2, ty)
            st["dh"] = st.pop("residual")
            if st["dh"] is not None:   # what comes down the residual stream
                st["dh"] *= 5e-3
            # what the forward pass left for the backward
            st["rstd"] = (st["x"].double().square().mean(1) + EPS).rsqrt().float()
        return st
    if op in ("quantize", "dequantize"):
        x = _activation(g, rows, dim)
        if case["pad"]:   # one position in sixteen is padding
            x *= torch.rand((rows, 1), generator=g, device=DEV) >= 1 / 16
        if op == "quantize":
            st["x"] = x.to(DT[ty])
        else:
            st["q"], st["s"] = _to8(x)
        return st
    if op == "weight":
        st["x"] = _randn(g, (rows, dim), 0.02, ty)
        return st
    st["q"], st["s"] = _to8(_activation(g, case["tokens"], dim))
    if op == "matmul":
        st["wq"], st["ws"] = _square8(_randn(g, (rows, dim), 0.02, F32))
        return st
    st["dy"] = _randn(g, (case["tokens"], rows), 1e-3, ty)
    st["G"] = torch.empty((rows, dim), device=DEV, dtype=DT[ty])   # the optimizer's gradient
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain(st):
    op = st["op"]
    if op in ("norm", "norm8"):
        x = st["x"]
        h = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
        f = h.float()
        rstd = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
        y = f * rstd * st["w"]
        out = _to8(y) if op == "norm8" else (y.to(x.dtype),)
        return (*out, h, rstd[:, 0])
    if op == "norm_bwd":
        x, rstd = st["x"].float(), st["rstd"][:, None]
        dy = st["dy"].float()
        xh, g = x * rstd, dy * st["w"]
        dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return dx.to(st["x"].dtype), (dy * xh).sum(0)
    if op == "quantize":
        return _to8(st["x"].float())
    if op == "dequantize":
        return _from8(st["q"], st["s"]).to(st["type"])
    if op == "weight":
        q, s = _square8(st["x"].float())
        return q, s, q.t().contiguous(), s.t().contiguous()
    x = _from8(st["q"], st["s"])
    if op == "matmul":
        return (x @ _from8(st["wq"], st["ws"], B).t()).to(st["type"])
    return (st["dy"].float().t() @ x).to(st["type"])


def _own(st):
    import matrix_optimizers_amd as mo
    op = st["op"]
    if op == "norm":
        return mo.rms_norm_forward(st["x"], st["w"], residual=st["residual"], eps=EPS)
    if op == "norm8":
        return mo.rms_norm_quantize(st["x"], st["w"], residual=st["residual"], eps=EPS)
    if op == "norm_bwd":
        return mo.rms_norm_backward(st["dy"], st["x"], st["rstd"], st["w"], dH=st["dh"])
    if op == "quantize":
        return mo.fp8_quantize(st["x"])
    if op == "dequantize":
        return mo.fp8_dequantize(st["q"], st["s"], dtype=st["type"])
    if op == "weight":
        return mo.fp8_quantize_weight(st["x"])
    if op == "matmul":
        return mo.fp8_matmul(st["q"], st["s"], st["wq"], st["ws"], dtype=st["type"])
    return mo.fp8_weight_grad(st["dy"], st["q"], st["s"], st["G"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the least a pass has to move and compute
# ---------------------------------------------------------------------------

def work(case):
    op, rows, dim = case["op"], case["rows"], case["dim"]
    es = 2 if case["type"] == BF16 else 4
    n, kb = rows * dim, -(-dim // B)
    if op == "norm_bwd":
        return {"bytes": (4 if case["residual"] else 3) * n * es + 8 * dim + 4 * rows, "flops": 10 * n}
    if op.startswith("norm"):
        out = n + rows * kb if op == "norm8" else n * es
        return {"bytes": (3 if case["residual"] else 1) * n * es + out + 4 * dim + 4 * rows, "flops": 6 * n}
    if op in ("quantize", "dequantize"):
        return {"bytes": n * (es + 1) + rows * kb, "flops": 2 * n}
    if op == "weight":
        return {"bytes": n * (es + 2) + 2 * -(-rows // B) * kb, "flops": 2 * n}
    t = case["tokens"]
    x = t * (dim + kb)
    if op == "matmul":
        return {"bytes": x + n + -(-rows // B) * kb + t * rows * es, "flops": 2 * t * n}
    return {"bytes": x + t * rows * es + n * es, "flops": 2 * t * n}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _grid(v):
    """v on e4m3's numbers: four significant bits, steps of 2^-9 below 2^-6, ties to even."""
    top = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(top - 3)
    return torch.round(v / step) * step


def _exponent(peak):
    e = torch.ceil(torch.log2(peak / 448))
    # where the logarithm or the power rounded
    e = e + (peak > 448 * torch.exp2(e)).double() - (peak <= 448 * torch.exp2(e - 1)).double()
    return torch.where(peak > 0, e, -127.0).clamp(min=-127)


def _exact8(v):
    rows, cols = v.shape
    peak = torch.stack([v[:, c:c + B].abs().amax(1) for c in range(0, cols, B)], 1)
    s = torch.exp2(_exponent(peak))
    at = torch.arange(cols, device=DEV) // B
    return _grid(v / s[:, at]), s


def _value(q, s, r=1):
    i, j = torch.arange(q.shape[0], device=DEV) // r, torch.arange(q.shape[1], device=DEV) // B
    return q.double() * s.double()[i][:, j]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm8", "norm_bwd"):
        return _exact_norm(st, op)
    if op == "quantize":
        parts = [_exact8(x.double()) for x in st["x"].split(max(1, (1 << 26) // case["dim"]))]
        return tuple(torch.cat(p) for p in zip(*parts))
    if op == "dequantize":
        return _value(st["q"], st["s"])
    if op == "weight":
        x = st["x"].double()
        rows, cols = x.shape
        peak = torch.stack([torch.stack([x[r:r + B, c:c + B].abs().max() for c in range(0, cols, B)])
                            for r in range(0, rows, B)])
        s = torch.exp2(_exponent(peak))
        i, j = torch.arange(rows, device=DEV) // B, torch.arange(cols, device=DEV) // B
        q = _grid(x / s[i][:, j])
        return q, s, q.t().contiguous(), s.t().contiguous()
    x = _value(st["q"], st["s"])
    if op == "matmul":
        return torch.mm(x, _value(st["wq"], st["ws"], B).t())
    return torch.mm(st["dy"].double().t(), x)


def _exact_norm(st, op):
    dim = st["x"].shape[1]
    step = max(1, (1 << 25) // dim)
    w = st["w"].double()
    parts, dw = [], torch.zeros_like(w)
    for r in range(0, st["x"].shape[0], step):
        rows = slice(r, r + step)
        x = st["x"][rows].double()
        if op == "norm_bwd":
            inv, dy = st["rstd"][rows].double()[:, None], st["dy"][rows].double()
            along = (dy * w * x).sum(1, keepdim=True) / dim
            dx = inv * (dy * w) - inv ** 3 * along * x
            dw += (dy * inv * x).sum(0)
            parts.append((dx if st["dh"] is None else dx + st["dh"][rows].double(),))
            continue
        total = x if st["residual"] is None else x + st["residual"][rows].double()
        h = total.to(st["x"].dtype).double()   # what is normed is what is stored
        inv = (h.square().sum(1) / dim + EPS) ** -0.5
        y = h * inv[:, None] * w
        parts.append((*(_exact8(y) if op == "norm8" else (y,)), total, inv))
    out = tuple(torch.cat(p) for p in zip(*parts))
    return (*out, dw) if op == "norm_bwd" else out
