"""Cases of the 8-bit and grouped operators, for measuring them.

Four operators: the root-mean-square norm with the residual's addition and
its 8-bit output (and its gradient), the quantiser to 8-bit floating point
with a scale for each block of 128, the 8-bit product of such operands, and
the products grouped by expert (16-bit inputs: forward, the two gradients;
8-bit inputs: forward).  `run` computes a case in plain torch operations, or,
with `own` set, through this package's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-5
BLOCK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
T16 = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the norm before a layer while one token is generated: latency
        {"name": "norm, one token", "op": "norm", "m": 1, "n": 4096, "t": "bf16"},
        # the same over a long prompt: bandwidth
        {"name": "norm, prompt", "op": "norm", "m": 8192, "n": 8192, "t": "bf16"},
        # its gradient in a training step, with the residual path's gradient
        {"name": "norm backward", "op": "norm_back", "m": 8190, "n": 5000, "t": "bf16"},
        # a step's output gradient, quantised along its rows
        {"name": "quantise rows", "op": "quant", "m": 16384, "n": 2048, "t": "bf16", "f": "e5m2", "rows": 1, "flip": False, "pow2": False},
        # a weight for the product with its transpose: square blocks, transposed
        {"name": "quantise weight transposed", "op": "quant", "m": 4000, "n": 8192, "t": "f32", "f": "e4m3", "rows": 128, "flip": True, "pow2": True},
        # one token through a linear layer: the weight's bytes and latency
        {"name": "f8 product, one token", "op": "f8", "m": 1, "n": 8192, "k": 4096, "fa": "e4m3", "rows": 128, "d": "bf16", "c": False},
        # a prompt through a linear layer: tensor throughput
        {"name": "f8 product, prompt", "op": "f8", "m": 8192, "n": 8192, "k": 4096, "fa": "e4m3", "rows": 128, "d": "bf16", "c": False},
        # a weight's gradient, both operands scaled along their rows, added to
        # the gradient so far; the reduction is over an odd number of tokens
        {"name": "f8 product, weight gradient", "op": "f8", "m": 2048, "n": 4096, "k": 8200, "fa": "e5m2", "rows": 1, "d": "f32", "c": True},
        # tokens sorted by expert through the experts' first layer
        {"name": "grouped forward", "op": "grouped", "t": "bf16", "tokens": 16384, "e": 32, "n": 4096, "k": 2048, "d": "bf16"},
        # the gradient of those tokens
        {"name": "grouped input gradient", "op": "grouped_in", "t": "bf16", "tokens": 16384, "e": 32, "n": 2048, "k": 4096, "d": "bf16"},
        # the gradient of the experts' weights
        {"name": "grouped weight gradient", "op": "grouped_w", "t": "bf16", "tokens": 16384, "e": 32, "n": 4096, "k": 2048, "d": "f32"},
        # a few generated tokens, spread over many experts: the weights' bytes
        {"name": "grouped f8, few tokens", "op": "grouped_f8", "tokens": 96, "e": 64, "n": 2048, "k": 4096, "d": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "quant", "f8", "f8", "grouped", "grouped_in", "grouped_w", "grouped_f8"])
    t = rng.choice(["bf16", "bf16", "f16"])
    if op in ("norm", "norm_back", "quant"):
        n = _log(rng, 256, 16384)
        m = _log(rng, 1, min(16384, 60_000_000 // n))
        if rng.random() < 0.5:
            n = -(-n // 64) * 64
        if op != "quant":
            return {"op": op, "m": m, "n": n, "t": t}
        return {"op": op, "m": m, "n": n, "t": rng.choice(["bf16", "f16", "f32"]), "f": rng.choice(["e4m3", "e5m2"]),
                "rows": rng.choice([1, 128]), "flip": rng.random() < 0.5, "pow2": rng.random() < 0.5}
    n, k = _log(rng, 256, 8192), _log(rng, 256, 8192)
    if rng.random() < 0.5:
        n, k = -(-n // 128) * 128, -(-k // 128) * 128
    if op == "f8":
        return {"op": op, "m": _log(rng, 1, min(8192, int(2.5e11 / (n * k)))), "n": n, "k": k, "fa": rng.choice(["e4m3", "e5m2"]),
                "rows": rng.choice([1, 128, 128]), "d": rng.choice(["bf16", "f16", "f32"]), "c": rng.random() < 0.3}
    e = _log(rng, 2, min(64, max(2, 250_000_000 // (n * k))))
    tokens = _log(rng, 1, min(16384, int(1.2e11 / (n * k))))
    d = rng.choice(["same", "f32"])
    case = {"op": op, "tokens": tokens, "e": e, "n": n, "k": k, "d": "bf16" if op == "grouped_f8" else t if d == "same" else "f32"}
    return case if op == "grouped_f8" else dict(case, t=t)


# ------------------------------------------------------------------- inputs

def _counts(case):
    """Tokens of each expert: uneven, as a router gives them, some without any."""
    rng = random.Random(case["tokens"] * 1000003 + case["e"] * 8191 + case["n"])
    share = [rng.lognormvariate(0.0, 0.7) for _ in range(case["e"])]
    share = [0.0 if rng.random() < 0.06 else s for s in share]
    if not sum(share):
        share[0] = 1.0
    got = [0] * case["e"]
    for i in rng.choices(range(case["e"]), share, k=case["tokens"]):
        got[i] += 1
    return got


def _offsets(case, seed):
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _rows(g, m, n, dtype, spread=1.0):
    """An m x n matrix whose rows start on 16-byte boundaries."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    wide = -(-n // per) * per
    x = torch.randn(m, wide, generator=g, device="cuda") * spread
    return x.to(dtype)[:, :n]


def _padded(q):
    """The same values in rows that start on 16-byte boundaries."""
    *lead, n = q.shape
    per = 16 // q.element_size()
    wide = torch.zeros(*lead, -(-n // per) * 16, dtype=torch.uint8, device=q.device).view(q.dtype)
    wide[..., :n] = q
    return wide[..., :n]


def _by_block(s):
    """Scales stored block after block, as the quantiser and the norm store them."""
    return s.transpose(-1, -2).contiguous().transpose(-1, -2)


def _uneven(g, m, n):
    """Values as activations have them: rows and some columns of other sizes."""
    x = torch.randn(m, n, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda"))
    x *= torch.exp(0.7 * torch.randn(1, n, generator=g, device="cuda"))
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_back"):
        t = T16[case["t"]]
        m, n = case["m"], case["n"]
        s["w"] = (1.0 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(t)
        s["x"] = _padded(_uneven(g, m, n).to(t))
        s["r"] = _rows(g, m, n, t, 2.0 if op == "norm" else 0.01)
        if op == "norm_back":
            s["dy"] = _rows(g, m, n, t, 0.01)
        return s
    if op == "quant":
        s["x"] = _padded(_uneven(g, case["m"], case["n"]).to(T16[case["t"]]))
        return s
    n, k = case["n"], case["k"]
    if op == "f8":
        m = case["m"]
        s["a"], s["sa"] = _quantise(_uneven(g, m, k), case["fa"], 1, False)
        s["b"], s["sb"] = _quantise(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k), "e4m3", case["rows"], False)
        s["a"], s["b"], s["sa"], s["sb"] = _padded(s["a"]), _padded(s["b"]), _by_block(s["sa"]), _by_block(s["sb"])
        s["c"] = _rows(g, m, n, T16[case["d"]]) if case["c"] else None
        return s
    at = _offsets(case, seed)
    e, tokens = case["e"], case["tokens"]
    s["most"] = max(b - a for a, b in zip(at, at[1:]))
    s["at"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    if op == "grouped_f8":
        s["a"], s["sa"] = _quantise(_uneven(g, tokens, k), "e4m3", 1, False)
        s["a"], s["sa"] = _padded(s["a"]), _by_block(s["sa"])
        w, sw = zip(*(_quantise(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k), "e4m3", 128, False) for _ in range(e)))
        s["b"], s["sb"] = _padded(torch.stack([x.view(torch.uint8) for x in w]).view(F8["e4m3"])), _by_block(torch.stack(sw))
        return s
    t = T16[case["t"]]
    if op == "grouped_w":
        s["dy"], s["x"] = _rows(g, tokens, n, t, 0.05), _rows(g, tokens, k, t)
        return s
    s["a"] = _rows(g, tokens, k, t)
    shape = (e, n, k) if op == "grouped" else (e, k, n)  # row-major: k x n
    w = torch.randn(*shape, generator=g, device="cuda") / math.sqrt(k)
    s["b"] = _padded(w.to(t))
    return s


# --------------------------------------------------------------- plain form

def _scale(most, f, pow2):
    """The scale of a block whose largest magnitude is `most`: that over the
    format's largest value, at least the smallest normal number; with pow2
    rounded up to a power of two."""
    s = torch.clamp(most / F8_MAX[f], min=2.0 ** -126)
    if pow2:
        frac, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(frac == 0.5, e - 1, e))
    return s


def _quantise(x, f, rows, pow2):
    m, n = x.shape
    mb = -(-m // rows)
    x = torch.nn.functional.pad(x.float(), (0, blocks(n) * BLOCK - n, 0, mb * rows - m)).view(mb, rows, blocks(n), BLOCK)
    s = _scale(x.abs().amax(dim=(1, 3), keepdim=True), f, pow2)
    q = torch.clamp(x / s, -F8_MAX[f], F8_MAX[f]).to(F8[f])
    return q.reshape(mb * rows, blocks(n) * BLOCK)[:m, :n], s.view(mb, blocks(n))


def _wide(q, s, rows):
    """The values that 8-bit q and its scales stand for, in 32 bits."""
    m, n = q.shape[-2:]
    s = s.repeat_interleave(rows, -2)[..., :m, :].repeat_interleave(BLOCK, -1)[..., :n]
    return q.float() * s


def _places(at, tokens, most):
    """Each token's place where every expert has `most` rows."""
    t = torch.arange(tokens, device=at.device)
    e = torch.searchsorted(at[1:].long(), t, right=True)
    return e * most + t - at.long()[e]


def _spread(x, at, e, most):
    p = torch.zeros(e * most, x.shape[1], device=x.device)
    p[_places(at, x.shape[0], most)] = x
    return p.view(e, most, -1)


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = s["x"].float() + s["r"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
        q, sc = _quantise(y, "e4m3", 1, False)
        return {"q": q, "s": sc, "h": h.to(s["x"].dtype)}
    if op == "norm_back":
        h, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        g = dy * w
        dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True))) + s["r"].float()
        return {"dx": dx.to(s["x"].dtype), "dw": (dy * h * r).sum(0)}
    if op == "quant":
        x = s["x"].t() if s["flip"] else s["x"]
        q, sc = _quantise(x, s["f"], s["rows"], s["pow2"])
        return {"q": q, "s": sc}
    d = T16[s["d"]]
    if op == "f8":
        y = _wide(s["a"], s["sa"], 1) @ _wide(s["b"], s["sb"], s["rows"]).t()
        return (y if s["c"] is None else y + s["c"].float()).to(d)
    e, most, at = s["e"], s["most"], s["at"]
    if op == "grouped_w":
        return torch.bmm(_spread(s["dy"].float(), at, e, most).transpose(1, 2), _spread(s["x"].float(), at, e, most)).to(d)
    if op == "grouped_f8":
        a, b = _wide(s["a"], s["sa"], 1), _wide(s["b"], s["sb"], 128).transpose(1, 2)
    else:
        a, b = s["a"].float(), s["b"].float()
        b = b.transpose(1, 2) if op == "grouped" else b
    y = torch.bmm(_spread(a, at, e, most), b).view(e * most, -1)
    return y[_places(at, a.shape[0], most)].to(d)


# -------------------------------------------------------------- own kernels

def _own(s):
    import mixed_precision_dense_02_gb300 as mma

    op = s["op"]
    if op == "norm":
        q, sc, h = mma.rmsnorm_f8(s["x"], s["w"], s["r"], eps=EPS)
        return {"q": q, "s": sc, "h": h}
    if op == "norm_back":
        dx, dw = mma.rmsnorm_backward(s["dy"], s["x"], s["w"], s["r"], eps=EPS)
        return {"dx": dx, "dw": dw}
    if op == "quant":
        q, sc = mma.quantize_f8(s["x"], fmt=s["f"], block_rows=s["rows"], transpose=s["flip"], pow2=s["pow2"])
        return {"q": q, "s": sc}
    d = T16[s["d"]]
    if op == "f8":
        return mma.gemm_f8(s["a"], s["sa"], s["b"], s["sb"], s["c"], out_dtype=d)
    if op == "grouped_w":
        return mma.gemm_grouped_wgrad(s["dy"], s["x"], s["at"], out_dtype=d)
    if op == "grouped_f8":
        return mma.gemm_grouped_f8(s["a"], s["sa"], s["b"], s["sb"], s["at"], out_dtype=d)
    return mma.gemm_grouped(s["a"], s["b"], s["at"], b_layout="col" if op == "grouped" else "row", out_dtype=d)


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------- exact, work

def exact(case, seed):
    """The definitions in 64 bits.  An 8-bit output has the value that was
    rounded to it."""
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64

    def amax(y, f, rows, pow2):
        m, n = y.shape
        out = torch.zeros(-(-m // rows), blocks(n), dtype=D, device=y.device)
        for j in range(blocks(n)):
            col = y[:, j * BLOCK:(j + 1) * BLOCK].abs().max(1).values
            if rows > 1:
                col = torch.cat([col, col.new_zeros(-m % rows)]).view(-1, rows).max(1).values
            out[:, j] = col
        out = (out / F8_MAX[f]).clamp_min(2.0 ** -126)
        return torch.pow(2.0, torch.ceil(torch.log2(out) - 1e-9)) if pow2 else out

    def over(y, sc, rows):
        rows_of = torch.arange(y.shape[0], device=y.device) // rows
        cols_of = torch.arange(y.shape[1], device=y.device) // BLOCK
        return y / sc[rows_of][:, cols_of]

    def values(q, sc, rows):
        rows_of = torch.arange(q.shape[0], device=q.device) // rows
        cols_of = torch.arange(q.shape[1], device=q.device) // BLOCK
        return q.to(D) * sc.to(D)[rows_of][:, cols_of]

    if op == "norm":
        h = s["x"].to(D) + s["r"].to(D)
        y = s["w"].to(D) * h / torch.sqrt((h ** 2).sum(1, keepdim=True) / case["n"] + EPS)
        sc = amax(y, "e4m3", 1, False)
        return {"q": over(y, sc, 1), "s": sc, "h": h}
    if op == "norm_back":
        h, dy, w = s["x"].to(D), s["dy"].to(D), s["w"].to(D)
        r = 1.0 / torch.sqrt((h ** 2).sum(1, keepdim=True) / case["n"] + EPS)
        n = h * r
        g = dy * w
        return {"dx": r * (g - n * ((g * n).sum(1, keepdim=True) / case["n"])) + s["r"].to(D), "dw": torch.einsum("mn,mn->n", dy, n)}
    if op == "quant":
        y = s["x"].to(D).t().contiguous() if case["flip"] else s["x"].to(D)
        sc = amax(y, case["f"], case["rows"], case["pow2"])
        return {"q": over(y, sc, case["rows"]), "s": sc}
    if op == "f8":
        y = torch.einsum("mk,nk->mn", values(s["a"], s["sa"], 1), values(s["b"], s["sb"], case["rows"]))
        return y if s["c"] is None else y + s["c"].to(D)
    at = s["at"].tolist()
    parts = []
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if op == "grouped_w":
            parts.append(torch.einsum("tn,tk->nk", s["dy"][a:b].to(D), s["x"][a:b].to(D)))
        elif op == "grouped_f8":
            parts.append(torch.einsum("tk,nk->tn", values(s["a"][a:b], s["sa"][a:b], 1), values(s["b"][e], s["sb"][e], 128)))
        else:
            parts.append(torch.einsum("tk,nk->tn" if op == "grouped" else "tk,kn->tn", s["a"][a:b].to(D), s["b"][e].to(D)))
    return torch.stack(parts) if op == "grouped_w" else torch.cat(parts)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back", "quant"):
        m, n, t = case["m"], case["n"], SIZE[case["t"]]
        if op == "norm":  # x, residual, weight; sum, 8 bits, scales
            return {"bytes": m * n * (3 * t + 1) + n * t + m * blocks(n) * 4, "flops": 8 * m * n}
        if op == "norm_back":  # dy, h, residual's gradient, weight; dx, dw
            return {"bytes": m * n * 4 * t + n * (t + 4), "flops": 12 * m * n}
        p, q = (n, m) if case["flip"] else (m, n)
        return {"bytes": m * n * (t + 1) + -(-p // case["rows"]) * blocks(q) * 4, "flops": 3 * m * n}
    n, k, d = case["n"], case["k"], SIZE[case["d"]]
    if op == "f8":
        m = case["m"]
        scales = 4 * blocks(k) * (m + -(-n // case["rows"]))
        return {"bytes": (m + n) * k + scales + m * n * d * (2 if case["c"] else 1), "flops": 2 * m * n * k}
    tokens, e = case["tokens"], case["e"]
    used = sum(c > 0 for c in _counts(case))
    flops = 2 * tokens * n * k
    if op == "grouped_w":
        return {"bytes": tokens * (n + k) * 2 + e * n * k * d + 4 * (e + 1), "flops": flops}
    if op == "grouped_f8":
        return {"bytes": (tokens + used * n) * k + 4 * blocks(k) * (tokens + used * blocks(n)) + tokens * n * d + 4 * (e + 1), "flops": flops}
    return {"bytes": (tokens + used * n) * k * 2 + tokens * n * d + 4 * (e + 1), "flops": flops}
