"""The router of a layer of experts and its gradient, against the definitions in 64
bits.

Tolerances.  CUDA's __expf of a distance d to the row's largest logit is within 2 +
1.173 |d| units in the last place, so within 2^-23 (2.5 + 1.2 |d|) relative; sums
over a row take at most 37 additions in a row and a division, below 2^-18; R is the
probabilities' mean of the first plus 2^-18.  A probability is within both of them
for its own d and R.  Sums over the tokens take at most 2^7 additions in a row per
warp, block and part: 2^-17.
Choices, their order and their numbers are compared exactly.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def rnd(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def logits(seed, t, e, dtype, ties=False, pad=0, gone=0.0):
    x = 2 * rnd(seed, t, e)
    if ties:
        x = (x * 2).round() / 2
    if gone:
        x = torch.where(rnd(seed + 9, t, e).abs() < gone, torch.full_like(x, -float("inf")), x)
    big = torch.full((t, e + pad), float("nan"), dtype=dtype, device="cuda")
    big[:, :e] = x.to(dtype)
    return big[:, :e]


def softmax(x):
    """(p, distances to the largest) in 64 bits; p is 0 in a row without experts."""
    top = x.amax(1, keepdim=True)
    d = torch.where(x == -float("inf"), torch.zeros_like(x), top - x).nan_to_num(0.0, 0.0, 0.0)
    p = torch.exp(x - top).nan_to_num(0.0)
    return p / p.sum(1, keepdim=True).clamp_min(1e-300), d


def want(x, k, mask, normalize):
    """All outputs in 64 bits, with the tolerances of weights and share."""
    t, e = x.shape
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask
    p, d = softmax(x)
    p = p * live[:, None]
    unit = 2.0 ** -23 * (2.5 + 1.2 * d)
    rel = unit + (p * unit).sum(1, keepdim=True) + 2.0 ** -18
    best = torch.sort(x, dim=1, descending=True, stable=True)
    chosen = torch.where(live[:, None] & (best.values[:, :k] > -float("inf")), best.indices[:, :k], -1)
    at = chosen.clamp(min=0)
    w = torch.where(chosen < 0, 0.0, p.gather(1, at))
    w_rel = rel.gather(1, at)
    if normalize:
        total = w.sum(1, keepdim=True)
        w_rel = w_rel + (w * w_rel).sum(1, keepdim=True) / total.clamp_min(1e-300)
        w = w / total.clamp_min(1e-300)
    ids = torch.where(chosen < 0, e, chosen).reshape(-1)
    order = torch.argsort(ids, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel())
    counts = torch.bincount(ids, minlength=e + 1)[:e]
    n = int(live.sum())
    share = p.sum(0) / max(n, 1)
    return {"weights": w, "w_rel": w_rel, "experts": chosen, "order": order, "place": place.view(t, k),
            "offsets": torch.nn.functional.pad(counts.cumsum(0), (1, 0)), "share": share,
            "share_tol": (p * (rel + 2.0 ** -17)).sum(0) / max(n, 1), "loss": e * (counts / max(n * k, 1) * share).sum(),
            "tokens": n, "counts": counts, "p": p, "rel": rel}


def check(got, ref, e, k):
    for name in ("experts", "order", "place", "offsets"):
        assert torch.equal(getattr(got, name).cpu().long(), ref[name]), name
    assert int(got.tokens) == ref["tokens"]
    err = (got.weights.double().cpu() - ref["weights"]).abs()
    assert bool((err <= ref["weights"] * ref["w_rel"] + 2.0 ** -126).all()), float((err / ref["weights"].clamp_min(1e-300)).max())
    tol = ref["share_tol"] + 2.0 ** -126
    assert bool(((got.share.double().cpu() - ref["share"]).abs() <= tol).all())
    lim = e * float((ref["counts"] / max(ref["tokens"] * k, 1) * (tol + 2.0 ** -17 * ref["share"])).sum()) + 2.0 ** -100
    assert abs(float(got.loss) - float(ref["loss"])) <= lim


SIZES = [(1, 1, 1), (1, 64, 6), (3, 7, 7), (5, 1024, 32), (63, 33, 2), (64, 32, 1), (65, 100, 8), (96, 64, 6), (97, 64, 6), (8, 1024, 3), (9, 1024, 3), (4864, 40, 3), (4865, 40, 3),
         (256, 300, 4), (257, 64, 8), (1000, 16, 2), (1000, 1000, 10), (4096, 256, 8), (20000, 8, 2),
         (20001, 130, 5), (300, 512, 32), (40000, 5, 1)]


@pytest.mark.parametrize("t,e,k", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_routes(t, e, k, kind):
    x = logits(t * 7 + e, t, e, T[kind], pad=e % 3)
    check(mma.route(x, k), want(x.double().cpu(), k, None, True), e, k)


@pytest.mark.parametrize("t,e,k", [(5, 40, 6), (200, 64, 8), (256, 512, 3), (700, 64, 8), (3000, 260, 12), (20000, 32, 4)])
@pytest.mark.parametrize("normalize", [True, False])
def test_masks_ties_and_missing_experts(t, e, k, normalize):
    x = logits(t + e, t, e, torch.float32, ties=True, gone=0.5)
    x[0] = -float("inf")  # a token without any expert
    x[1, 2:] = -float("inf")  # with fewer than k
    x[2 % t, :] = 1.0  # all equal
    x[3 % t] = x[3 % t] * 0.0  # zeros of either sign
    x[3 % t, 1::2] = -x[3 % t, 1::2].abs()
    x[3 % t].nan_to_num_(0.0)
    mask = (rnd(t, t) > -0.5).cuda()
    got = mma.route(x, k, mask=mask, normalize=normalize)
    check(got, want(x.double().cpu(), k, mask.cpu(), normalize), e, k)
    none = torch.zeros(t, dtype=torch.bool, device="cuda")
    got = mma.route(x, k, mask=none, normalize=normalize)
    check(got, want(x.double().cpu(), k, none.cpu(), normalize), e, k)
    assert float(got.loss) == 0 and bool((got.experts == -1).all())


@pytest.mark.parametrize("t", [40, 1000])
def test_bad_logits_stay_with_their_token(t):
    e, k = 70, 5
    x = logits(1, t, e, torch.float32)
    clean = want(x.double().cpu(), k, None, True)
    x[7, 3], x[11, 60], x[13] = float("nan"), float("inf"), -float("nan")
    got = mma.route(x, k)
    assert bool(got.weights[[7, 11, 13]].isnan().all()) and bool(got.share.isnan().any()) and bool(got.loss.isnan())
    assert bool(((got.experts >= 0) & (got.experts < e)).all())
    keep = torch.ones(t, dtype=torch.bool)
    keep[[7, 11, 13]] = False
    assert torch.equal(got.experts.cpu().long()[keep], clean["experts"][keep])
    assert torch.equal(torch.sort(got.order).values.cpu().long(), torch.arange(t * k))
    assert torch.equal(got.place.reshape(-1)[got.order.long()].cpu().long(), torch.arange(t * k))


def test_no_tokens():
    got = mma.route(torch.empty(0, 16, device="cuda"), 4)
    assert got.weights.shape == (0, 4) and not got.offsets.any() and not got.share.any() and float(got.loss) == 0
    assert mma.route_backward(torch.empty(0, 16, device="cuda"), got).shape == (0, 16)


def want_back(x, k, mask, normalize, dw, dl):
    r = want(x, k, mask, normalize)
    t, e = x.shape
    n = max(r["tokens"], 1)
    p, rel = r["p"], r["rel"] + 2.0 ** -18
    live = torch.ones(t, 1) if mask is None else mask[:, None]
    a = (dl * e / (n * n * k)) * r["counts"].double()[None, :].expand(t, e)
    at, has = r["experts"].clamp(min=0), (r["experts"] >= 0).double()
    w = r["weights"]
    if normalize:
        dot = (p * a).sum(1, keepdim=True)
        g = w * has * (dw - (w * dw).sum(1, keepdim=True))
        dx = (p * (a - dot)).scatter_add(1, at, g)
        mag = p * (a.abs() + (p * a.abs()).sum(1, keepdim=True))
        gm = w * has * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
        w_rel = r["w_rel"] + 2.0 ** -18
        worst = (rel + (p * rel).sum(1, keepdim=True)) * mag
        # (a weight's error reaches the sum over the chosen: at most the largest of them)
        worst = worst.scatter_add(1, at, gm * (w_rel + w_rel.amax(1, keepdim=True)))
    else:
        d = a.scatter_add(1, at, dw * has)
        dm = a.abs().scatter_add(1, at, dw.abs() * has)
        dx = p * (d - (p * d).sum(1, keepdim=True))
        worst = p * (rel + rel.amax(1, keepdim=True)) * (dm + (p * dm).sum(1, keepdim=True))
    return dx * live, worst * live


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 64, 6), (65, 100, 8), (300, 512, 32), (1000, 1000, 10), (5000, 256, 8), (20001, 13, 2)])
@pytest.mark.parametrize("kind,normalize,masked,which", [
    ("f32", True, False, "both"), ("f32", False, True, "both"), ("bf16", True, True, "weights"),
    ("f16", False, False, "loss"), ("f32", True, True, "loss"), ("bf16", False, False, "weights"), ("f32", True, False, "none")])
def test_gradient(t, e, k, kind, normalize, masked, which):
    x = logits(t + 3 * e, t, e, T[kind], pad=1, gone=0.3 if e > 8 else 0.0)
    mask = (rnd(t, t) > -0.7).cuda() if masked else None
    dw = rnd(t + 1, t, k).float().cuda() if which in ("both", "weights") else None
    dl = torch.tensor(37.0, device="cuda") if which in ("both", "loss") else None
    r = mma.route(x, k, mask=mask, normalize=normalize)
    got = mma.route_backward(x, r, dw, dl, mask=mask, normalize=normalize)
    ref, worst = want_back(x.double().cpu(), k, None if mask is None else mask.cpu(), normalize,
                           torch.zeros(t, k, dtype=torch.float64) if dw is None else dw.double().cpu(),
                           0.0 if dl is None else 37.0)
    err = (got.double().cpu() - ref).abs()
    lim = (ref.abs() + worst) * U[kind] + worst + TINY[kind]
    assert got.dtype == T[kind] and bool((err <= lim).all()), float((err / lim).max())


def test_gradient_against_differences():
    """A loss of the weights and the balance loss along a random direction, the
    choices fixed by wide gaps.  A central difference of step 2^-6 is off by about
    step^2 / 6 of the third derivative, below 2^-12 of the slope's scale, and by
    rounding, 2^-22 / step = 2^-16 of the loss's scale."""
    t, e, k, step = 40, 12, 3, 2.0 ** -6
    x = torch.stack([torch.randperm(e, generator=torch.Generator().manual_seed(i)).double() / 3 for i in range(t)])
    dw, dl = rnd(3, t, k), 2.0
    for normalize in (True, False):
        def loss(x):
            r = mma.route(x.float().cuda(), k, normalize=normalize)
            return float((r.weights.double().cpu() * dw).sum()) + dl * float(r.loss)
        x0 = x.float().cuda()
        g = mma.route_backward(x0, mma.route(x0, k, normalize=normalize), dw.float().cuda(),
                               torch.tensor(dl, device="cuda"), normalize=normalize).double().cpu()
        for seed in (1, 2, 3):
            d = rnd(seed, t, e).clamp(-2, 2)
            slope = (loss(x + step * d) - loss(x - step * d)) / (2 * step)
            assert abs(slope - float((g * d).sum())) <= 2.0 ** -10 * float((g * d).abs().sum()) + 2.0 ** -14 * (dw.abs().sum() + 4)


def test_two_streams_and_graphs():
    x = [logits(i, 3000 + i, 64, torch.float32) for i in range(2)]
    alone = [mma.route(v, 4) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        together = [mma.route(v, 4, stream=s) for v, s in zip(x, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    still, dw = x[0].clone(), torch.ones(3000, 4, device="cuda")
    dl = torch.ones((), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mma.route(still, 4)
        d = mma.route_backward(still, r, dw, dl)
    for seed in (5, 6):
        still.copy_(logits(seed, 3000, 64, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        again = mma.route(still, 4)
        assert all(torch.equal(p, q) for p, q in zip(r, again))
        assert torch.equal(d, mma.route_backward(still, again, dw, dl))
