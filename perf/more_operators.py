"""Cases of the layer norm, the router and the products with low-rank adapters,
for measuring them.

Three families: the layer norm with the residual's addition (16-bit or 8-bit
output) and its gradient; the router of a layer of experts (the best k of a
token's logits, their weights, the tokens sorted by expert, a balance loss) and
its gradient; and products in which every request's rows have a low-rank
adapter of their own beside the shared matrix, with their gradients.  `run`
computes a case in plain torch operations, or, with `own` set, through this
package's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-5
BLOCK = 128
F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the norm before a layer while one token is generated: latency
        {"name": "layer norm, one token", "op": "norm", "m": 1, "n": 4096, "t": "bf16", "f8": False, "bias": True, "res": True},
        # the same over a long prompt, for 8-bit products: bandwidth
        {"name": "layer norm, prompt in 8 bits", "op": "norm", "m": 8192, "n": 8192, "t": "bf16", "f8": True, "bias": True, "res": True},
        # its gradient in a training step, with the residual path's gradient
        {"name": "layer norm backward", "op": "norm_back", "m": 8190, "n": 5000, "t": "bf16", "res": True},
        # a few generated tokens before a layer of experts: latency
        {"name": "route, generated tokens", "op": "route", "tokens": 96, "e": 64, "k": 6, "t": "f32", "mask": False, "norm": True},
        # a training batch before a layer of many experts, with padding
        {"name": "route, training batch", "op": "route", "tokens": 16384, "e": 256, "k": 8, "t": "f32", "mask": True, "norm": True},
        # the gradient of its logits, of the balance loss and of the weights
        {"name": "route backward", "op": "route_back", "tokens": 16384, "e": 256, "k": 8, "t": "f32", "mask": True, "norm": True},
        # one request's token through a linear layer: latency, the weight's bytes
        {"name": "adapters, one token", "op": "lora", "t": "bf16", "tokens": 1, "single": 1, "requests": 1, "adapters": 4, "n": 8192, "k": 4096, "r": 16, "d": "bf16"},
        # a token each of many requests: the weight's and the adapters' bytes
        {"name": "adapters, 64 requests' tokens", "op": "lora", "t": "bf16", "tokens": 64, "single": 64, "requests": 64, "adapters": 64, "n": 8192, "k": 4096, "r": 16, "d": "bf16"},
        # a serving step with a few prompts and many requests' tokens
        {"name": "adapters, prompts and tokens", "op": "lora", "t": "f16", "tokens": 2100, "single": 60, "requests": 63, "adapters": 40, "n": 4096, "k": 4096, "r": 32, "d": "f16"},
        # long prompts, or a training batch of several adapters: tensor throughput
        {"name": "adapters, prompts", "op": "lora", "t": "bf16", "tokens": 8192, "single": 0, "requests": 6, "adapters": 8, "n": 8192, "k": 4096, "r": 64, "d": "bf16"},
        # the gradient of that batch's input
        {"name": "adapters, input gradient", "op": "lora_in", "t": "bf16", "tokens": 8192, "single": 0, "requests": 6, "adapters": 8, "n": 4096, "k": 8192, "r": 64, "d": "bf16"},
        # the gradient of its adapters
        {"name": "adapters, their gradient", "op": "lora_w", "t": "bf16", "tokens": 8192, "single": 0, "requests": 6, "adapters": 8, "n": 8192, "k": 4096, "r": 16, "d": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "route", "route", "route_back", "lora", "lora", "lora", "lora_in", "lora_w"])
    t = rng.choice(["bf16", "bf16", "f16"])
    if op in ("norm", "norm_back"):
        n = _log(rng, 256, 16384)
        m = _log(rng, 1, min(16384, 60_000_000 // n))
        if rng.random() < 0.5:
            n = -(-n // 64) * 64
        case = {"op": op, "m": m, "n": n, "t": rng.choice(["bf16", "f16", "f32"]), "res": rng.random() < 0.6}
        return case if op == "norm_back" else dict(case, f8=rng.random() < 0.5, bias=rng.random() < 0.7)
    if op in ("route", "route_back"):
        e = _log(rng, 4, 512)
        return {"op": op, "tokens": _log(rng, 1, 16384), "e": e, "k": min(e, rng.randint(1, 8)), "t": rng.choice(["f32", "f32", "bf16", "f16"]),
                "mask": rng.random() < 0.4, "norm": rng.random() < 0.7}
    n, k = _log(rng, 256, 8192), _log(rng, 256, 8192)
    if rng.random() < 0.5:
        n, k = -(-n // 128) * 128, -(-k // 128) * 128
    tokens = _log(rng, 1, min(8192, int(2.5e11 / (n * k))))
    single = min(tokens, rng.choice([0, 0, tokens, rng.randint(0, 64)]))
    long = min(tokens - single, rng.randint(1, 8))
    r = rng.choice([8, 16, 16, 32, 64, rng.randint(1, 128)])
    return {"op": op, "t": t, "tokens": tokens, "single": single if long else tokens, "requests": (single if long else tokens) + long,
            "adapters": rng.randint(1, 48), "n": n, "k": k, "r": r, "d": rng.choice([t, t, "f32"])}


# ------------------------------------------------------------------- inputs

def _lengths(case):
    """Rows of each request: single tokens, and prompts of uneven lengths."""
    rng = random.Random(case["tokens"] * 1000003 + case["requests"] * 8191 + case["n"])
    long = case["requests"] - case["single"]
    got = [1] * case["requests"]
    share = [rng.lognormvariate(0.0, 0.6) for _ in range(long)]
    for i in rng.choices(range(long), share, k=case["tokens"] - case["requests"]) if long else ():
        got[i] += 1
    return got


def _chosen(case):
    """The requests' adapters: some share one, some have none (-1)."""
    rng = random.Random(case["tokens"] * 7919 + case["requests"] * 31 + case["r"])
    return [-1 if rng.random() < 0.06 and case["requests"] > 1 else rng.randrange(case["adapters"]) for _ in range(case["requests"])]


def _aligned(x, dtype):
    """x rounded to dtype, in rows that start on 16-byte boundaries."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    wide = torch.zeros(*x.shape[:-1], -(-x.shape[-1] // per) * per, dtype=dtype, device=x.device)
    wide[..., :x.shape[-1]] = x
    return wide[..., :x.shape[-1]]


def _uneven(g, m, n):
    """Values as activations have them: rows and some columns of other sizes,
    some columns far from zero."""
    x = torch.randn(m, n, generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(1, n, generator=g, device="cuda"))
    x += 0.5 * torch.randn(1, n, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda"))
    return x


def _logits(g, case):
    x = 1.5 * torch.randn(case["tokens"], case["e"], generator=g, device="cuda")
    x += 0.5 * torch.randn(1, case["e"], generator=g, device="cuda")
    return _aligned(x, TYPES[case["t"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op in ("norm", "norm_back"):
        t = TYPES[case["t"]]
        m, n = case["m"], case["n"]
        s["w"] = (1.0 + 0.1 * randn(n)).to(t)
        s["x"] = _aligned(_uneven(g, m, n), t)
        s["r"] = _aligned(randn(m, n) * (1.0 if op == "norm" else 0.01), t) if case["res"] else None
        if op == "norm":
            s["b"] = (0.1 * randn(n)).to(t) if case["bias"] else None
        else:
            s["dy"] = _aligned(0.01 * randn(m, n), t)
        return s
    if op in ("route", "route_back"):
        s["x"] = _logits(g, case)
        s["live"] = None
        if case["mask"]:  # sequences of a batch, padded at their ends
            tokens = case["tokens"]
            length = max(1, tokens // 8)
            at = torch.arange(tokens, device="cuda")
            ends = torch.randint(length // 2, length + 1, (tokens // length + 1,), generator=g, device="cuda")
            s["live"] = at % length < ends[at // length]
        if op == "route_back":
            s["dw"] = 0.01 * randn(case["tokens"], case["k"])
            s["dl"] = torch.full((), 0.01, device="cuda")
            s["route"] = _route(s)
            if own:
                import mixed_precision_dense_02_gb300 as mma

                s["kept"] = mma.Routing(**s["route"])
        return s
    t = TYPES[case["t"]]
    tokens, n, k, r, many = case["tokens"], case["n"], case["k"], case["r"], case["adapters"]
    plan = list(zip(_lengths(case), _chosen(case)))
    random.Random(seed).shuffle(plan)
    at = [0]
    for rows, _ in plan:
        at.append(at[-1] + rows)
    s["plan"] = [(a, b, c) for a, b, (_, c) in zip(at, at[1:], plan)]
    s["at"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    s["of"] = torch.tensor([c for _, c in plan], dtype=torch.int32, device="cuda")
    s["x"] = _aligned(randn(tokens, k), t)
    if op == "lora_w":
        s["dy"] = _aligned(0.05 * randn(tokens, n), t)
        none = torch.tensor([c < 0 for _, _, c in s["plan"]], device="cuda").repeat_interleave((s["at"][1:] - s["at"][:-1]).long())[:, None]
        s["s"] = randn(tokens, r).masked_fill(none, 0.0)
        s["u"] = (0.05 * randn(tokens, r)).masked_fill(none, 0.0)
        return s
    s["scale"] = torch.rand(many, generator=g, device="cuda") + 0.5
    if op == "lora":
        s["w"] = _aligned(randn(n, k) / math.sqrt(k), t)
        s["a"] = _aligned(randn(many, r, k) / math.sqrt(k), t)
        s["b"] = _aligned(randn(many, n, r) / math.sqrt(4 * r), t)
    else:  # stored with the result's columns side by side
        s["w"] = _aligned(randn(k, n) / math.sqrt(k), t)
        s["a"] = _aligned(randn(many, k, r) / math.sqrt(k), t)
        s["b"] = _aligned(randn(many, r, n) / math.sqrt(4 * r), t)
    return s


# --------------------------------------------------------------- plain form

def _quantise(y):
    m, n = y.shape
    y = torch.nn.functional.pad(y, (0, blocks(n) * BLOCK - n)).view(m, blocks(n), BLOCK)
    s = torch.clamp(y.abs().amax(dim=2, keepdim=True) / F8_MAX, min=2.0 ** -126)
    q = torch.clamp(y / s, -F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
    return q.reshape(m, -1)[:, :n], s.view(m, -1)


def _norm(s):
    x = s["x"].float()
    h = x if s["r"] is None else x + s["r"].float()
    c = h - h.mean(1, keepdim=True)
    y = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    t = s["x"].dtype
    out = {"h": h.to(t)} if s["r"] is not None else {}
    if s["f8"]:
        q, sc = _quantise(y)
        return dict(out, q=q, s=sc)
    return dict(out, y=y.to(t))


def _norm_back(s):
    h, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    c = h - h.mean(1, keepdim=True)
    r = torch.rsqrt(c.square().mean(1, keepdim=True) + EPS)
    xh = c * r
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _softmax(x):
    p = torch.exp(x - x.max(1, keepdim=True).values)
    return p / p.sum(1, keepdim=True)


def _route(s):
    x, k, live = s["x"].float(), s["k"], s["live"]
    tokens, e = x.shape
    p = _softmax(x)
    chosen = torch.sort(x, stable=True, dim=1, descending=True).indices[:, :k]
    w = p.gather(1, chosen)
    if s["norm"]:
        w = w / w.sum(1, keepdim=True)
    if live is not None:
        p, w = p * live[:, None], w * live[:, None]
        chosen = torch.where(live[:, None], chosen, -1)
    flat = torch.where(chosen < 0, e, chosen).reshape(-1)
    order = torch.argsort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=x.device).scatter_add_(0, flat, torch.ones_like(flat))[:e]
    n = torch.full((), tokens, device=x.device) if live is None else live.sum()
    share = p.sum(0) / n.clamp(min=1)
    loss = e * (counts.float() * share).sum() / (n * k).clamp(min=1)
    return {"weights": w, "experts": chosen.int(), "order": order.int(), "place": place.view(tokens, k).int(),
            "offsets": torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int(), "share": share, "loss": loss, "tokens": n.int()}


def _route_back(s):
    x, k, live, got = s["x"].float(), s["k"], s["live"], s["route"]
    e = x.shape[1]
    p = _softmax(x)
    n = got["tokens"].float().clamp(min=1)
    counts = (got["offsets"][1:] - got["offsets"][:-1]).float()
    d = (e * s["dl"] / (n * n * k)) * counts[None, :].expand_as(p)
    at = got["experts"].long().clamp(min=0)
    if s["norm"]:
        w, dw = got["weights"], s["dw"]
        dx = p * (d - (p * d).sum(1, keepdim=True))
        dx = dx.scatter_add(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        d = d.scatter_add(1, at, s["dw"])
        dx = p * (d - (p * d).sum(1, keepdim=True))
    if live is not None:
        dx = dx * live[:, None]
    return dx.to(s["x"].dtype)


def _lora(s):
    x, row = s["x"].float(), s["op"] == "lora_in"
    w = s["w"].float()
    y = x @ (w if row else w.t())
    for i, j, c in s["plan"]:
        if c >= 0:
            a, b = s["a"][c].float(), s["b"][c].float()
            y[i:j] += s["scale"][c] * ((x[i:j] @ (a if row else a.t())) @ (b if row else b.t()))
    return y.to(TYPES[s["d"]])


def _lora_w(s):
    x, dy = s["x"].float(), s["dy"].float()
    da = torch.zeros(s["adapters"], s["r"], s["k"], device=x.device)
    db = torch.zeros(s["adapters"], s["n"], s["r"], device=x.device)
    for i, j, c in s["plan"]:
        if c >= 0:
            da[c] += s["u"][i:j].t() @ x[i:j]
            db[c] += dy[i:j].t() @ s["s"][i:j]
    d = TYPES[s["d"]]
    return {"da": da.to(d), "db": db.to(d)}


_PLAIN = {"norm": _norm, "norm_back": _norm_back, "route": _route, "route_back": _route_back, "lora": _lora, "lora_in": _lora, "lora_w": _lora_w}


# -------------------------------------------------------------- own kernels

def _own(s):
    import mixed_precision_dense_02_gb300 as mma

    op = s["op"]
    if op == "norm":
        if s["f8"]:
            q, sc, h = mma.layernorm_f8(s["x"], s["w"], s["b"], s["r"], eps=EPS)
            out = {"q": q, "s": sc}
        else:
            y, h = mma.layernorm(s["x"], s["w"], s["b"], s["r"], eps=EPS)
            out = {"y": y}
        return out if s["r"] is None else {"h": h, **out}
    if op == "norm_back":
        dx, dw, db = mma.layernorm_backward(s["dy"], s["x"], s["w"], s["r"], eps=EPS)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "route":
        return mma.route(s["x"], s["k"], mask=s["live"], normalize=s["norm"])._asdict()
    if op == "route_back":
        return mma.route_backward(s["x"], s["kept"], s["dw"], s["dl"], mask=s["live"], normalize=s["norm"])
    if op == "lora_w":
        da, db = mma.gemm_lora_wgrad(s["dy"], s["x"], s["s"], s["u"], s["at"], s["of"], adapters_total=s["adapters"], out_dtype=TYPES[s["d"]])
        return {"da": da, "db": db}
    return mma.gemm_lora(s["x"], s["w"], s["a"], s["b"], s["at"], s["of"], s["scale"], b_layout="col" if op == "lora" else "row", out_dtype=TYPES[s["d"]])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# -------------------------------------------------------------- exact, work

def exact(case, seed):
    """The definitions in 64 bits.  An 8-bit output has the value that was
    rounded to it."""
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64

    if op == "norm":
        h = s["x"].to(D) + (0.0 if s["r"] is None else s["r"].to(D))
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        y = (h - mean) / torch.sqrt(var + EPS) * s["w"].to(D) + (0.0 if s["b"] is None else s["b"].to(D))
        out = {} if s["r"] is None else {"h": h}
        if not case["f8"]:
            return dict(out, y=y)
        sc = torch.stack([y[:, j * BLOCK:(j + 1) * BLOCK].abs().max(1).values for j in range(blocks(case["n"]))], 1)
        sc = (sc / F8_MAX).clamp_min(2.0 ** -126)
        return dict(out, q=y / sc[:, torch.arange(case["n"], device=y.device) // BLOCK], s=sc)
    if op == "norm_back":
        h, g = s["x"].to(D), s["dy"].to(D) * s["w"].to(D)
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        std = torch.sqrt(var + EPS)
        z = (h - mean) / std
        n = case["n"]
        dx = (n * g - g.sum(1, keepdim=True) - z * torch.einsum("mn,mn->m", g, z)[:, None]) / (n * std)
        return {"dx": dx if s["r"] is None else dx + s["r"].to(D), "dw": torch.einsum("mn,mn->n", s["dy"].to(D), z), "db": s["dy"].to(D).sum(0)}
    if op in ("route", "route_back"):
        x, k = s["x"].to(D), case["k"]
        tokens, e = x.shape
        live = torch.ones(tokens, dtype=torch.bool, device=x.device) if s["live"] is None else s["live"]
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) * live[:, None]
        # the k best, one after the other; of equal ones the first
        left, best = x.clone(), []
        for _ in range(k):
            top = (left == left.max(1, keepdim=True).values).int().argmax(1)
            best.append(top)
            left[torch.arange(tokens, device=x.device), top] = -math.inf
        best = torch.stack(best, 1)
        w = torch.gather(p, 1, best)
        if case["norm"]:
            w = torch.where(live[:, None], w / w.sum(1, keepdim=True), 0.0)
        n, ids = int(live.sum()), torch.where(live[:, None], best, e).reshape(-1)
        counts = torch.bincount(ids, minlength=e + 1)[:e]
        share = p.sum(0) / max(n, 1)
        if op == "route":
            order = torch.sort(ids * (tokens * k) + torch.arange(tokens * k, device=x.device)).values % (tokens * k)
            offsets = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
            offsets[1:] = torch.cumsum(counts, 0)
            return {"weights": w, "experts": torch.where(live[:, None], best, -1).int(), "order": order.int(),
                    "place": torch.argsort(order).view(tokens, k).int(), "offsets": offsets, "share": share,
                    "loss": e * torch.dot(counts.to(D) / max(n * k, 1), share), "tokens": torch.tensor(n, dtype=torch.int32, device=x.device)}
        a = s["dl"].to(D) * e * counts.to(D) / (max(n, 1) ** 2 * k)
        d = a.expand(tokens, e).clone()
        if case["norm"]:
            # w_j = p_j / sum of the chosen p: by p_j (dw_j - sum of w dw) / that sum
            total = p.gather(1, best).sum(1, keepdim=True).clamp_min(1e-300)
            d.scatter_add_(1, best, (s["dw"].to(D) - torch.einsum("tk,tk->t", w, s["dw"].to(D))[:, None]) / total)
        else:
            d.scatter_add_(1, best, s["dw"].to(D))
        return p * (d - torch.einsum("te,te->t", p, d)[:, None])
    if op == "lora_w":
        da = torch.zeros(case["adapters"], case["r"], case["k"], dtype=D, device="cuda")
        db = torch.zeros(case["adapters"], case["n"], case["r"], dtype=D, device="cuda")
        for c in set(c for _, _, c in s["plan"] if c >= 0):
            rows = torch.cat([torch.arange(i, j, device="cuda") for i, j, o in s["plan"] if o == c])
            da[c] = torch.einsum("tr,tk->rk", s["u"][rows].to(D), s["x"][rows].to(D))
            db[c] = torch.einsum("tn,tr->nr", s["dy"][rows].to(D), s["s"][rows].to(D))
        return {"da": da, "db": db}
    flip = op == "lora_in"
    x = s["x"].to(D)
    y = torch.matmul(x, s["w"].to(D) if flip else s["w"].to(D).t())
    for c in set(c for _, _, c in s["plan"] if c >= 0):
        rows = torch.cat([torch.arange(i, j, device="cuda") for i, j, o in s["plan"] if o == c])
        low = torch.einsum("tk,kr->tr" if flip else "tk,rk->tr", x[rows], s["a"][c].to(D)) * s["scale"][c].to(D)
        y[rows] += torch.einsum("tr,rn->tn" if flip else "tr,nr->tn", low, s["b"][c].to(D))
    return y


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        m, n, t = case["m"], case["n"], SIZE[case["t"]]
        if op == "norm":  # x, residual and their sum, the output, weight and bias
            out = m * n + 4 * m * blocks(n) if case["f8"] else m * n * t
            return {"bytes": m * n * t * (3 if case["res"] else 1) + out + n * t * (2 if case["bias"] else 1), "flops": 9 * m * n}
        # dy, h, residual's gradient, weight; dx, dw, db
        return {"bytes": m * n * t * (4 if case["res"] else 3) + n * (t + 8), "flops": 15 * m * n}
    if op in ("route", "route_back"):
        tokens, e, k, t = case["tokens"], case["e"], case["k"], SIZE[case["t"]]
        mask = tokens if case["mask"] else 0
        if op == "route":  # logits; weights, experts, order, place; offsets, share
            return {"bytes": tokens * (e * t + 16 * k) + mask + 8 * e, "flops": tokens * e * (4 + k)}
        # logits, weights and their gradient, experts, offsets; the gradient
        return {"bytes": tokens * (2 * e * t + 12 * k) + mask + 4 * e, "flops": 8 * tokens * e}
    tokens, n, k, r, d = case["tokens"], case["n"], case["k"], case["r"], SIZE[case["d"]]
    chosen = _chosen(case)
    rows = sum(m for m, c in zip(_lengths(case), chosen) if c >= 0)
    used = len(set(chosen) - {-1})
    index = 4 * (2 * case["requests"] + 1)
    if op == "lora_w":
        return {"bytes": rows * (2 * (n + k) + 8 * r) + case["adapters"] * r * (n + k) * d + index, "flops": 2 * rows * r * (n + k)}
    return {"bytes": 2 * (tokens * k + n * k + used * r * (n + k)) + tokens * n * d + 4 * used + index,
            "flops": 2 * tokens * n * k + 2 * rows * r * (n + k)}
