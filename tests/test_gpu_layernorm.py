"""The layer norm, its 8-bit output and its gradient, against the definitions in
64 bits.

Tolerances.  An FP32 sum of a row runs over at most 64 terms per thread, ten
levels of a tree and 32 warps, each addition off by 2^-24 of a partial sum, so a
mean is within 106 * 2^-24 < 2^-17 of the mean magnitude that it sums (`far`:
that over the row's deviation).  The deviation inherits 2^-17 and, where a term
is a distance to the mean, far * 2^-17; five more roundings are below 2^-20.  So
z = c / std is within 2^-16 (1 + far) (1 + |z|), and the result, z w + b, is
rounded once more (2^-24 of each, and half a step of its type).
The gradient's terms are sums of such products; each is bounded by its
magnitudes times 2^-15 (1 + far).  A column's sum over the rows takes at most
2^8 additions in a row per block or part: 2^-16 of its magnitudes.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half an ulp
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -127}  # half the smallest step


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


def rows16(x, dtype, pad=0):
    """x on the GPU with rows on 16-byte boundaries, `pad` more 16-byte chunks
    between them, and NaN in the gaps."""
    m, n = x.shape
    per = 16 // torch.empty((), dtype=dtype).element_size()
    big = torch.full((m, -(-n // per) * per + pad * per), float("nan"), dtype=dtype, device="cuda")
    big[:, :n] = x.to(dtype)
    return big[:, :n]


def host(t):
    return t.double().cpu()


def centred(h, eps):
    """(z, std, far) of rows h in 64 bits."""
    c = h - h.mean(1, keepdim=True)
    std = (c.square().mean(1, keepdim=True) + eps).sqrt()
    return c / std, std, h.abs().mean(1, keepdim=True) / std


def want_y(h, w, b, eps):
    z, _, far = centred(h, eps)
    y = z * w + b
    return y, 2.0 ** -16 * (1 + far) * (1 + z.abs()) * w.abs() + 2.0 ** -22 * (y.abs() + b.abs())


SHAPES = [(1, 1), (1, 7), (3, 8), (1, 4096), (5, 100), (200, 264), (160, 2048), (400, 2056), (7, 4100),
          (300, 5000), (170, 8192), (33, 8190), (3, 16384), (155, 16384), (2, 16392), (3, 40000), (400, 9001),
          (300, 16400), (5, 60000)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", SHAPES)
def test_forward(m, n, t):
    seed = m * 131 + n
    res, bias, w32 = (m + n) % 2 == 0, n % 3 != 0, m % 2 == 0
    x = rows16(rnd(seed, m, n) + 3 * rnd(seed + 1, m, 1), T[t], pad=m % 3)
    r = rows16(rnd(seed + 2, m, n), T[t], pad=1) if res else None
    wt = torch.float32 if w32 else T[t]
    w = (1 + 0.3 * rnd(seed + 3, n)).to(wt).cuda()
    b = rnd(seed + 4, n).to(wt).cuda() if bias else None
    y, h = mma.layernorm(x, w, b, r, eps=1e-5)
    total = host(x) + (host(r) if res else 0)
    if res:
        # (the FP32 sum is itself rounded, by 2^-24 of it)
        assert bool(((host(h) - total).abs() <= total.abs() * (U[t] + 2.0 ** -23) + TINY[t]).all())
    else:
        assert h is x
    want, tol = want_y(total, host(w), host(b) if bias else torch.zeros(n, dtype=torch.float64), 1e-5)
    err = (host(y) - want).abs()
    bound = (want.abs() + tol) * U[t] + tol + TINY[t]
    assert bool((err <= bound).all()), float((err / bound).max())
    again, _ = mma.layernorm(x, w, b, r, eps=1e-5)
    assert torch.equal(y, again)


@pytest.mark.parametrize("m,n,t,pow2", [(1, 4096, "bf16", False), (70, 1000, "bf16", True), (9, 8190, "f16", False),
                                        (200, 392, "f32", False), (2, 20000, "bf16", False), (3, 9000, "f32", True)])
def test_8_bit_output(m, n, t, pow2):
    x, r = rows16(rnd(n, m, n) + 1, T[t]), rows16(rnd(n + 1, m, n), T[t])
    w, b = (1 + 0.3 * rnd(n + 2, n)).to(T[t]).cuda(), rnd(n + 3, n).to(T[t]).cuda()
    q, s, h, y = mma.layernorm_f8(x, w, b, r, pow2=pow2, y=True)
    y1, h1 = mma.layernorm(x, w, b, r)
    assert torch.equal(y, y1) and torch.equal(h, h1)
    want, tol = want_y(host(x) + host(r), host(w), host(b), 1e-5)
    blocks = -(-n // 128)
    pad = torch.nn.functional.pad
    top = pad(want.abs(), (0, blocks * 128 - n)).view(m, blocks, 128).amax(2) / 448
    slack = pad(tol, (0, blocks * 128 - n)).view(m, blocks, 128).amax(2) / 448
    sh = host(s)
    if pow2:
        assert bool((torch.log2(sh) == torch.log2(sh).round()).all())
        assert bool((sh >= (top - slack) * (1 - 2.0 ** -22)).all()) and bool((sh < 2 * (top + slack) * (1 + 2.0 ** -22)).all())
    else:
        assert bool(((sh - top).abs() <= slack + top * 2.0 ** -22).all())
    of = sh.repeat_interleave(128, 1)[:, :n]
    v = want / of
    # half a step of E4M3 (2^-4 of a normal number, 2^-10 below), of the quotient
    # as computed
    off = tol / of + v.abs() * 2.0 ** -22
    bound = torch.maximum((v.abs() + off) * 2.0 ** -4, torch.tensor(2.0 ** -10)) + off
    err = (host(q) - v).abs()
    # (a value above 448 by the scale's rounding is the largest one)
    assert bool((err <= bound).all()), float((err / bound).max())


def want_back(dy, h, w, r, eps):
    z, std, far = centred(h, eps)
    g = dy * w
    n = h.shape[1]
    gm, gz = g.mean(1, keepdim=True), (g * z).mean(1, keepdim=True)
    dx = (g - gm - z * gz) / std + r
    k = 2.0 ** -15 * (1 + far)
    parts = g.abs() + g.abs().mean(1, keepdim=True)
    tol = k * (parts + (1 + z.abs()) * (1 + far) * (parts * (1 + z.abs())).mean(1, keepdim=True)) / std + 2.0 ** -23 * r.abs()
    dw, dw_tol = (dy * z).sum(0), (dy.abs() * (k * (1 + z.abs()) + 2.0 ** -16 * z.abs())).sum(0)
    return dx, tol, dw, dw_tol, dy.sum(0), 2.0 ** -16 * dy.abs().sum(0)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", SHAPES + [(1000, 520), (2000, 4096)])
def test_backward(m, n, t):
    seed = m * 17 + n
    res, w32 = (m + n) % 2 == 1, m % 2 == 1
    h = rows16(rnd(seed, m, n) + 2 * rnd(seed + 1, m, 1), T[t], pad=m % 2)
    dy = rows16(rnd(seed + 2, m, n), T[t])
    r = rows16(rnd(seed + 3, m, n), T[t], pad=2) if res else None
    w = (1 + 0.3 * rnd(seed + 4, n)).to(torch.float32 if w32 else T[t]).cuda()
    dx, dw, db = mma.layernorm_backward(dy, h, w, r, eps=1e-5)
    want, tol, dw64, dw_tol, db64, db_tol = want_back(host(dy), host(h), host(w), host(r) if res else torch.zeros(1, dtype=torch.float64), 1e-5)
    for name, got, ref, lim in (("dx", host(dx), want, (want.abs() + tol) * U[t] + tol + TINY[t]),
                                ("dw", host(dw), dw64, dw_tol + 2.0 ** -126), ("db", host(db), db64, db_tol + 2.0 ** -126)):
        err = (got - ref).abs()
        assert bool((err <= lim).all()), (name, float((err / lim).max()))
    again = mma.layernorm_backward(dy, h, w, r, eps=1e-5)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))


def test_gradient_against_differences():
    """The loss sum(dy * y) along random directions; FP32 inputs.  A central
    difference with step 2^-8 of a smooth function of O(1) scale is off by about
    step^2 = 2^-16 of it, and by 2^-24 * sqrt(n m) / step of rounding: 2^-9 of the
    derivative's scale covers both."""
    m, n, step = 6, 200, 2.0 ** -8
    h, dy, w, b = rnd(1, m, n), rnd(2, m, n), 1 + 0.3 * rnd(3, n), rnd(4, n)
    dev = lambda a: a.float().cuda()  # noqa: E731
    dx, dw, db = mma.layernorm_backward(dev(dy), dev(h), dev(w))

    def loss(h, w, b):
        return float((host(mma.layernorm(dev(h), dev(w), dev(b))[0]) * dy).sum())

    for got, args, of in ((dx, (h, w, b), 0), (dw, (h, w, b), 1), (db, (h, w, b), 2)):
        d = rnd(10 + of, *args[of].shape)
        up, down = list(args), list(args)
        up[of], down[of] = args[of] + step * d, args[of] - step * d
        slope = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(slope - float((host(got) * d).sum())) <= 2.0 ** -9 * float(host(got).norm() * d.norm()) + 2.0 ** -9


def test_rows_far_from_zero_and_bad_rows():
    n = 4096
    h = rnd(5, 8, n)
    h[1] += 1000.0
    h[2, 7] = float("inf")
    h[3, 9] = float("nan")
    h[4] = 5.0  # no deviation at all
    h[6] = 1e4 * h[6]
    for t in ("f32", "bf16"):
        x = rows16(h, T[t])
        one, zero = torch.ones(n, dtype=T[t], device="cuda"), torch.zeros(n, dtype=T[t], device="cuda")
        y, _ = mma.layernorm(x, one, zero)
        y = host(y)
        assert bool(y[2].isnan().all()) and bool(y[3].isnan().all())
        assert bool((y[4] == 0).all())
        good = [0, 1, 5, 6, 7]
        want, tol = want_y(host(x)[good], torch.ones(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64), 1e-5)
        assert bool(((y[good] - want).abs() <= (want.abs() + tol) * U[t] + tol).all())
        # in the gradient bad rows keep to themselves but for the columns' sums
        dx, _, db = mma.layernorm_backward(rows16(torch.ones_like(h), T[t]), x, one)
        dx = host(dx)
        assert bool(dx[2].isnan().all()) and bool(dx[[0, 1, 4, 5, 6, 7]].isfinite().all())
        assert bool((host(db) == 8).all())


def test_no_rows_and_in_place_and_streams():
    w = torch.ones(64, device="cuda")
    y, h = mma.layernorm(torch.empty(0, 64, device="cuda"), w)
    assert y.shape == (0, 64)
    dx, dw, db = mma.layernorm_backward(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"), w)
    assert not dw.any() and not db.any() and dx.shape == (0, 64)
    x = rows16(rnd(8, 300, 64), torch.float32)
    want = mma.layernorm(x, w)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mma.layernorm(x, w, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    # rows of the ABI's H over X itself
    r = rows16(rnd(9, 300, 64), torch.float32)
    keep, out = x.clone(), torch.empty_like(x)
    st = binding.load().mma_layernorm(6 - 1, 5, 300, 64, x.data_ptr(), 64, r.data_ptr(), 64, w.data_ptr(), None, 1e-5, 0,
                                      x.data_ptr(), 64, out.data_ptr(), 64, None, 0, None, 0, 0,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(x, keep + r)
    assert torch.equal(out, mma.layernorm(keep, w, None, r)[0])


@pytest.mark.parametrize("m,n", [(5, 264), (700, 264), (9, 8200), (500, 9000)])
def test_gradient_in_place(m, n):
    """The ABI's DX over DY, and over the residual's gradient."""
    h, w = rows16(rnd(1, m, n), torch.float32), torch.ones(n, device="cuda")
    dy, r = rows16(rnd(2, m, n), torch.float32), rows16(rnd(3, m, n), torch.float32)
    want = mma.layernorm_backward(dy, h, w, r)
    need = binding.load().mma_layernorm_backward_workspace(m, n)
    for over in range(2):
        d, g = dy.clone(), r.clone()
        dx = (d, g)[over]
        dw, db, ws = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")
        st = binding.load().mma_layernorm_backward(5, 5, m, n, d.data_ptr(), n, h.data_ptr(), n, w.data_ptr(), 1e-5, g.data_ptr(), n,
                                                   dx.data_ptr(), n, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need,
                                                   torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])


def test_captured_and_replayed():
    x, dy = rows16(rnd(11, 500, 1024), torch.bfloat16), rows16(rnd(12, 500, 1024), torch.bfloat16)
    w = torch.ones(1024, device="cuda", dtype=torch.bfloat16)
    mma.layernorm_backward(dy, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = mma.layernorm(x, w)
        grads = mma.layernorm_backward(dy, x, w)
    for seed in (13, 14):
        x.copy_(rnd(seed, 500, 1024))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mma.layernorm(x, w)[0])
        assert all(torch.equal(a, b) for a, b in zip(grads, mma.layernorm_backward(dy, x, w)))


@pytest.mark.parametrize("t,n", [("f32", 4096), ("bf16", 4096), ("f32", 5003), ("f16", 264), ("bf16", 10000)])
def test_many_rows_of_every_kind(t, n):
    """Rows in turn per block: far from zero, with the 32 elements that a row is
    sampled at far from the others, without deviation, with
    infinities.  The samples' mean is then far from the row's, and both the
    variance and the gradient's sums have to be those about the row's own mean."""
    m = 700
    h = rnd(n, m, n)
    q = n // 32
    at = torch.arange(32) * q + 2 * torch.arange(32) % q
    h[1::7] += 300.0
    for i in range(2, m, 7):
        h[i, at] += 1000.0
    h[3::7] = 0.0
    h[3::7, at[:9]] = 200.0
    h[4::7] = 7.0
    h[5::28, 3] = float("inf")
    h[12::28, n - 1] = float("nan")
    x = rows16(h, T[t])
    w, b = (1 + 0.3 * rnd(3, n)).to(T[t]).cuda(), rnd(4, n).to(T[t]).cuda()
    y, _ = mma.layernorm(x, w, b)
    bad = ~host(x).isfinite().all(1)
    assert bool(host(y)[bad].isnan().all())
    good = ~bad
    want, tol = want_y(host(x)[good], host(w), host(b), 1e-5)
    err = (host(y)[good] - want).abs()
    bound = (want.abs() + tol) * U[t] + tol
    assert bool((err <= bound).all()), float((err / bound).max())
    dy = rows16(rnd(5, m, n), T[t])
    dx, _, _ = mma.layernorm_backward(dy, x, w)
    assert bool(host(dx)[bad].isnan().all())
    flat = torch.zeros(m, dtype=torch.bool)
    flat[4::7] = True  # (no deviation: the factor is 1 / sqrt(eps), of rounded means)
    keep = good & ~flat
    want, tol, *_ = want_back(host(dy)[keep], host(x)[keep], host(w), torch.zeros(1, dtype=torch.float64), 1e-5)
    err = (host(dx)[keep] - want).abs()
    bound = (want.abs() + tol) * U[t] + tol
    assert bool((err <= bound).all()), float((err / bound).max())
    assert bool(host(dx)[good & flat].isfinite().all())
    # the weights' gradient over the rows without infinities
    rows = good.nonzero()[:, 0].cuda()
    xs, ds = rows16(host(x)[good], T[t]), rows16(host(dy)[good], T[t])
    _, dw, db = mma.layernorm_backward(ds, xs, w)
    _, _, dw64, dw_tol, db64, db_tol = want_back(host(ds), host(xs), host(w), torch.zeros(1, dtype=torch.float64), 1e-5)
    assert rows.numel() == xs.shape[0]
    assert bool(((host(dw) - dw64).abs() <= dw_tol).all()) and bool(((host(db) - db64).abs() <= db_tol).all())
