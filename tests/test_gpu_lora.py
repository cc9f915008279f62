"""Products with low-rank adapters of many requests, their input's gradient and the
adapters' gradients, against the definitions in 64 bits.

Tolerances.  A tensor core's FP32 sums are off by at most 2^-16 of the sum of the
terms' magnitudes at the lengths here (measured 4.2e-6 = 2^-17.9 at 4096 terms in a
row; the kernels add at most 1024 of them before they round to nearest).  The rows'
sums S inherit that from x A; in the second product S may be rounded to the inputs'
type, half a step U of it, or with an FP32 result to a sum of three BF16 numbers,
U^3, or two FP16 ones, U^2; the products with W and with B are off by another 2^-16 of their magnitudes, and the
result is rounded to its type.  FP16 numbers below 2^-14 have steps of 2^-24: half of
that for each S and, with two parts, for what the first leaves.
"""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
STEP = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
SUM = 2.0 ** -16


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
    """x on the GPU with rows on 16-byte boundaries, `pad` more 16-byte chunks between
    them, and NaN in the gaps."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    big = torch.full((*x.shape[:-1], -(-x.shape[-1] // per) * per + pad * per), float("nan"), dtype=dtype, device="cuda")
    big[..., :x.shape[-1]] = x.to(dtype)
    return big[..., :x.shape[-1]]


def host(t):
    return t.double().cpu()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Operands of a call and its values in 64 bits."""

    def __init__(self, lengths, n, k, r, adapters, total, kind="bf16", row=False, gap=(0, 0), scales=True, seed=0, pad=0):
        t = gap[0] + sum(lengths) + gap[1]
        self.t, self.n, self.k, self.r, self.kind, self.row, self.total = t, n, k, r, kind, row, total
        at = [gap[0]]
        for m in lengths:
            at.append(at[-1] + m)
        dt = T[kind]
        self.at, self.of = at, adapters
        self.offsets = ints(at)
        self.adapters = None if adapters is None else ints(adapters)
        self.x = rows16(rnd(seed, t, k), dt, pad)
        w, a, b = rnd(seed + 1, n, k) / k ** 0.5, rnd(seed + 2, total, r, k) / k ** 0.5, rnd(seed + 3, total, n, r) / r ** 0.5
        self.w = rows16(w.t() if row else w, dt, pad)
        self.a = rows16(a.transpose(1, 2) if row else a, dt)
        self.b = rows16(b.transpose(1, 2) if row else b, dt, pad)
        self.scales = (0.5 + rnd(seed + 4, total).abs()).float().cuda() if scales else None

    def who(self, j):
        a = j if self.of is None else self.of[j]
        return a if 0 <= a < self.total else -1

    def want(self):
        x, w, a, b = host(self.x), host(self.w), host(self.a), host(self.b)
        if self.row:
            w, a, b = w.t(), a.transpose(1, 2), b.transpose(1, 2)
        sc = torch.ones(self.total, dtype=torch.float64) if self.scales is None else host(self.scales)
        d, mag = x @ w.t(), SUM * (x.abs() @ w.abs().t())
        s, s_tol = torch.zeros(self.t, self.r, dtype=torch.float64), torch.zeros(self.t, self.r, dtype=torch.float64)
        up, u_in = torch.zeros_like(d), torch.zeros_like(d)
        for j, (i0, i1) in enumerate(zip(self.at, self.at[1:])):
            c = self.who(j)
            if c < 0 or i1 <= i0:
                continue
            s[i0:i1] = sc[c] * (x[i0:i1] @ a[c].t())
            s_tol[i0:i1] = SUM * sc[c] * (x[i0:i1].abs() @ a[c].abs().t())
            up[i0:i1] = s[i0:i1] @ b[c].t()
            mag[i0:i1] += s_tol[i0:i1] @ b[c].abs().t() + SUM * (s[i0:i1].abs() @ b[c].abs().t())
            u_in[i0:i1] = (s[i0:i1].abs() + s_tol[i0:i1]) @ b[c].abs().t() + 0.0
            self.half = STEP[self.kind] * b.abs().sum(2).max()
        return d + up, mag, u_in, s, s_tol

    def run(self, out, c=None, d=None, **kw):
        return mma.gemm_lora(self.x, self.w, self.a, self.b, self.offsets, self.adapters, self.scales, c, d,
                             b_layout="row" if self.row else "col", out_dtype=T[out], sums=True, **kw)

    def check(self, out, c=None, **kw):
        got, s = self.run(out, c, **kw)
        want, mag, u_in, s64, s_tol = self.want()
        u = U[self.kind]
        tol = mag + u_in * ((u ** 3 if self.kind == "bf16" else u * u) if out == "f32" else u) + getattr(self, "half", 0.0)
        if c is not None:
            want = want + host(c)
            tol = tol + 2.0 ** -23 * host(c).abs()
        lim = (want.abs() + tol) * U[out] + tol + STEP[out]
        err = (host(got) - want).abs()
        assert got.dtype == T[out] and bool((err <= lim).all()), float((err / lim).max())
        serr = (host(s) - s64).abs()
        assert bool((serr <= s_tol + 2.0 ** -23 * s64.abs() + 2.0 ** -140).all())
        return got, s


def random_lengths(seed, count, most):
    rng = random.Random(seed)
    return [rng.choice([0, 1, 1, 2, rng.randint(1, most)]) for _ in range(count)]


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("lengths,n,k,r", [
    ([1], 256, 512, 16), ([1, 1, 1], 200, 264, 8), ([5, 0, 7, 1], 136, 72, 1), ([1] * 32, 1000, 1024, 16),
    ([1] * 33, 264, 520, 24), ([64], 512, 4096, 64), ([1] * 64, 4104, 256, 7), ([3] * 40, 520, 136, 65),
    ([128], 130, 1000, 128), ([129], 256, 300, 16), ([200, 1, 1, 1, 30, 9, 8, 7], 776, 512, 32),
    ([700, 300], 1100, 264, 128), ([1] * 300, 264, 264, 16), ([9] * 90, 300, 520, 40),
    ([1] * 1024, 136, 264, 16), ([1] * 1025, 264, 136, 20), ([0] * 1500 + [3, 0, 40], 264, 264, 16),
    (([1, 0, 2] * 50 + [90] + [0] * 1000) * 4 + [1, 30], 300, 200, 33)])
def test_product(lengths, n, k, r, kind, out, row):
    rng = random.Random(n + k)
    total = max(1, min(len(lengths), 11))
    adapters = [rng.choice([-1, total + 3] + list(range(total)) * 4) for _ in lengths]
    Case(lengths, n, k, r, adapters, total, kind, row, gap=(rng.choice([0, 3]), rng.choice([0, 5])), seed=n, pad=n % 2).check(out)


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("t,out", [(3, "bf16"), (50, "f32"), (100, "bf16"), (600, "f32"), (600, "bf16")])
def test_addend_and_no_scales_and_own_adapters(t, out, row):
    lengths = random_lengths(t, 20, max(1, t // 6))
    case = Case(lengths, 328, 200, 12, None, 20, "bf16", row, scales=False, seed=t)
    c = rows16(rnd(t, case.t, 328), T[out], 1)
    want, _ = case.check(out, c)
    d = c.clone()
    got, _ = case.run(out, d, d)  # in place
    assert got.data_ptr() == d.data_ptr() and torch.equal(got, want)


def test_many_random_batches():
    for seed in range(30):
        rng = random.Random(seed)
        lengths = random_lengths(seed, rng.randint(1, 60), rng.choice([4, 40, 300]))
        total = rng.randint(1, 9)
        n, k, r = rng.randint(1, 700), rng.randint(1, 900), rng.choice([1, 8, 16, 33, 64, 100, 128])
        adapters = [rng.randint(-1, total) for _ in lengths]
        if sum(lengths) == 0:
            lengths[0] = 1
        Case(lengths, n, k, r, adapters, total, rng.choice(["bf16", "f16"]), rng.random() < 0.4,
             gap=(rng.randint(0, 2), rng.randint(0, 70)), seed=seed).check(rng.choice(["bf16", "f32"]) if rng.random() < 0 else "f32")


def test_no_requests_no_adapters_no_rank():
    x, w = rows16(rnd(1, 40, 64), T["bf16"]), rows16(rnd(2, 72, 64), T["bf16"])
    plain = mma.gemm_lora(x, w, rows16(rnd(3, 2, 8, 64), T["bf16"]), rows16(rnd(4, 2, 72, 8), T["bf16"]), ints([0]))
    want = (host(x) @ host(w).t())
    assert bool(((host(plain) - want).abs() <= want.abs() * 2.0 ** -8 + SUM * (host(x).abs() @ host(w).abs().t())).all())
    none, s = mma.gemm_lora(x, w, rows16(rnd(3, 2, 8, 64), T["bf16"]), rows16(rnd(4, 2, 72, 8), T["bf16"]), ints([0, 40]), ints([-1]), sums=True)
    assert torch.equal(none, plain) and not s.any()
    zero = torch.zeros(0, 8, 64, dtype=T["bf16"], device="cuda")
    assert torch.equal(mma.gemm_lora(x, w, zero, zero.new_zeros(0, 72, 8), ints([0, 40])), plain)
    thin = torch.zeros(2, 0, 64, dtype=T["bf16"], device="cuda")
    assert torch.equal(mma.gemm_lora(x, w, thin, thin.new_zeros(2, 72, 0), ints([0, 40])), plain)
    assert mma.gemm_lora(x[:0], w, rows16(rnd(3, 2, 8, 64), T["bf16"]), rows16(rnd(4, 2, 72, 8), T["bf16"]), ints([0, 0])).shape == (0, 72)


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("lengths", [[1, 3, 0, 2], [150, 1, 2, 40]])
def test_no_k(lengths, row):
    """Without k nothing is read of X, W and A, and the sums are zeros: the result is the addend."""
    t, n, r = T["bf16"], 328, 12
    m = sum(lengths)
    x, c = torch.empty(m, 0, dtype=t, device="cuda"), rows16(rnd(1, m, n), t)
    w = torch.empty((0, n) if row else (n, 0), dtype=t, device="cuda")
    a = torch.empty((4, 0, r) if row else (4, r, 0), dtype=t, device="cuda")
    b = rows16(rnd(2, 4, r, n) if row else rnd(2, 4, n, r), t)
    offsets = ints([0] + list(torch.tensor(lengths).cumsum(0)))
    d, s = mma.gemm_lora(x, w, a, b, offsets, C=c, b_layout="row" if row else "col", sums=True)
    assert torch.equal(d, c) and not s.any()
    # the ABI takes no matrices at all then
    need = binding.load().mma_gemm_lora_workspace(2, 2, m, n, r, 4)
    ws, s = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.ones(m, 16, device="cuda")
    d.zero_()
    assert c.stride(0) == d.stride(0) == n
    st = binding.load().mma_gemm_lora(2, 2, m, n, 0, r, None, 0, None, 0, None, 0, 0, None, 0, 0, 1 if row else 0, 4,
                                      offsets.data_ptr(), None, 4, None, c.data_ptr(), n, d.data_ptr(), n, s.data_ptr(), 16,
                                      ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(d, c) and not s[:, :r].any()


def test_most_requests():
    """As many as the call takes, most of them empty, and offsets that go back."""
    lengths = [0] * 65536
    for i in range(0, 65536, 701):
        lengths[i] = 1 + i % 5
    lengths[30000], lengths[65535] = 70, 2
    adapters = [(i // 3) % 8 - 1 for i in range(65536)]
    c = Case(lengths, 200, 136, 16, adapters, 7, "bf16", seed=2, gap=(3, 9))
    want, s = c.check("f32")
    dy, u = rows16(rnd(5, c.t, 200), T["bf16"]), rnd(7, c.t, 16).float().cuda()
    g = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=7)
    a64, b64, ma, mb = wgrad_want(c, dy, s, u)
    for got, ref, mag in zip(g, (a64, b64), (ma, mb)):
        tol = mag * (SUM + U["bf16"] ** 3) + 2.0 ** -20 * STEP["bf16"]
        assert bool(((host(got) - ref).abs() <= (ref.abs() + tol) * U["f32"] + tol + STEP["f32"]).all())
    good = c.offsets.clone()
    later = good.clone()
    later[40000:40010] -= 50  # raised to the one before
    later[0] = -3
    c.offsets = later
    low = torch.cummax(later.clamp(0, c.t), 0)[0]
    got, _ = c.run("f32")
    c.offsets = low
    assert torch.equal(got, c.run("f32")[0])
    h = [mma.gemm_lora_wgrad(dy, c.x, s, u, o, c.adapters, adapters_total=7) for o in (later, low)]
    assert torch.equal(h[0][0], h[1][0]) and torch.equal(h[0][1], h[1][1])


def test_offsets_out_of_range_and_order():
    """Clamped, and decreasing ones raised to the one before, as in grouped products."""
    good = Case([10, 0, 30, 20], 136, 128, 16, [0, 1, 2, 3], 4, seed=3)
    want = good.run("f32")
    bad = Case([10, 0, 30, 20], 136, 128, 16, [0, 1, 2, 3], 4, seed=3)
    bad.offsets = ints([-5, 10, 7, 40, 1000])
    got = bad.run("f32")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("lengths", [[1] * 12, [1, 1, 20, 30], [140, 160, 5, 1, 1]])
def test_bad_numbers_stay_with_their_adapter_and_row(lengths, row):
    case = Case(lengths, 264, 136, 16, list(range(len(lengths))), len(lengths), "bf16", row, seed=9)
    clean, s0 = case.run("bf16")
    case.a[1] = float("nan")
    case.b[2] = float("inf")
    case.x[0, 5] = float("inf")  # (the first request's first row)
    got, s = case.run("bf16")
    at = case.at
    keep = torch.ones(case.t, dtype=torch.bool)
    keep[0] = False
    keep[at[1]:at[3]] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep]) and torch.equal(s.cpu()[keep], s0.cpu()[keep])
    assert bool(got[at[1]:at[2]].isnan().all()) and not bool(got[at[2]:at[3]].isfinite().any())


def test_input_gradient_is_the_other_layout():
    """dX of the col call's D against the formula: the row call with A and B changed
    places, and its sums."""
    c = Case([300, 1, 1, 50], 256, 320, 16, [1, 0, -1, 2], 3, "bf16", seed=4)
    dy = rows16(rnd(8, c.t, 256), T["bf16"])
    dx, u = mma.gemm_lora(dy, c.w, c.b, c.a, c.offsets, c.adapters, c.scales, b_layout="row", out_dtype=T["f32"], sums=True)
    g, w, a, b, sc = host(dy), host(c.w), host(c.a), host(c.b), host(c.scales)
    want, tol = g @ w, SUM * (g.abs() @ w.abs())
    for j, (i0, i1) in enumerate(zip(c.at, c.at[1:])):
        q = c.who(j)
        if q >= 0:
            want[i0:i1] += sc[q] * ((g[i0:i1] @ b[q]) @ a[q])
            tol[i0:i1] += 3 * SUM * sc[q] * ((g[i0:i1].abs() @ b[q].abs()) @ a[q].abs())
    assert bool(((host(dx) - want).abs() <= tol + want.abs() * 2.0 ** -24).all())


def wgrad_want(c, dy, s, u):
    x, g = host(c.x), host(dy)
    da, db = torch.zeros(c.total, c.r, c.k, dtype=torch.float64), torch.zeros(c.total, c.n, c.r, dtype=torch.float64)
    ma, mb = torch.zeros_like(da), torch.zeros_like(db)
    for j, (i0, i1) in enumerate(zip(c.at, c.at[1:])):
        q = c.who(j)
        if q >= 0:
            da[q] += host(u)[i0:i1].t() @ x[i0:i1]
            db[q] += g[i0:i1].t() @ host(s)[i0:i1]
            ma[q] += host(u)[i0:i1].abs().t() @ x[i0:i1].abs()
            mb[q] += g[i0:i1].abs().t() @ host(s)[i0:i1].abs()
    return da, db, ma, mb


@pytest.mark.parametrize("kind,out", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("lengths,n,k,r", [
    ([1], 256, 512, 16), ([5, 0, 7, 1], 136, 72, 1), ([1] * 33, 264, 520, 24), ([700, 300], 1100, 264, 128),
    ([64, 65, 63], 200, 136, 64), ([2000], 128, 128, 8), ([300] * 9, 520, 392, 40), ([3] * 200, 144, 130, 12),
    ([1] * 1100, 136, 200, 16), ([2, 1] * 40 + [90], 264, 130, 65), (([1, 0, 2] * 50 + [90] + [0] * 1000) * 4 + [1, 30], 300, 200, 33)])
def test_adapters_gradient(lengths, n, k, r, kind, out):
    rng = random.Random(n * k)
    total = max(1, min(len(lengths), 7))
    adapters = [rng.choice([-1, total] + list(range(total)) * 4) for _ in lengths]
    c = Case(lengths, n, k, r, adapters, total, kind, gap=(rng.choice([0, 4]), rng.choice([0, 9])), seed=k)
    dy = rows16(rnd(5, c.t, n), T[kind], 1)
    s, u = rows16(rnd(6, c.t, r), torch.float32, 1), rnd(7, c.t, r).float().cuda()
    da, db = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=total, out_dtype=T[out])
    a64, b64, ma, mb = wgrad_want(c, dy, s, u)
    rel = SUM + (U[kind] ** (3 if kind == "bf16" else 2) if out == "f32" else U[kind])
    for got, ref, mag in ((da, a64, ma), (db, b64, mb)):
        tol = mag * rel + 2.0 ** -20 * STEP[kind]
        # (FP16 sums below 2^-14 have steps of 2^-24)
        tol = tol + (2.0 ** -25 * c.t * 5 if kind == "f16" else 0.0)
        lim = (ref.abs() + tol) * U[out] + tol + STEP[out]
        err = (host(got) - ref).abs()
        assert got.dtype == T[out] and bool((err <= lim).all()), float((err / lim).max())
    again = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=total, out_dtype=T[out])
    assert torch.equal(da, again[0]) and torch.equal(db, again[1])
    # added to what is there; adapters without rows keep theirs
    if out == "f32":
        a0, b0 = rnd(1, total, r, k).float().cuda(), rnd(2, total, n, r).float().cuda()
        a1, b1 = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=total, dA=a0.clone(), dB=b0.clone(), accumulate=True)
        assert torch.equal(a1, a0 + da) and torch.equal(b1, b0 + db)


def test_gradient_against_differences():
    """The loss sum(dy * D) along random directions of A and B, FP32 results: it is
    linear in each, so a central difference is off by rounding alone: 2^-8 of inputs
    that have to be numbers of BF16 is avoided by steps that are."""
    c = Case([130, 3, 1, 70], 136, 200, 16, [0, 1, 0, 2], 3, "bf16", seed=11)
    dy = rows16(rnd(12, c.t, 136).sign(), T["bf16"])
    _, s = c.run("f32")
    _, u = mma.gemm_lora(dy, c.w, c.b, c.a, c.offsets, c.adapters, c.scales, b_layout="row", sums=True)
    da, db = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=3)

    def loss():
        return float((host(c.run("f32")[0]) * host(dy)).sum())

    for m, g in ((c.a, da), (c.b, db)):
        keep = m.clone()
        for seed in (1, 2):
            step = rnd(seed, *m.shape).sign().to(T["bf16"]).cuda()
            m.copy_(step)
            up = loss()
            m.copy_(-step)
            down = loss()
            m.copy_(keep)
            slope = (up - down) / 2
            scale = float((host(g) * host(step)).abs().sum())
            assert abs(slope - float((host(g) * host(step)).sum())) <= 2.0 ** -12 * scale


def test_bad_numbers_stay_with_their_adapters_gradient():
    """Rows of one request with NaN and infinities, next to others inside a block."""
    lengths = [100, 30, 70, 300, 5]
    c = Case(lengths, 136, 200, 24, [0, 1, 2, 3, 4], 5, "bf16", seed=21)
    dy = rows16(rnd(5, c.t, 136), T["bf16"])
    s, u = rnd(6, c.t, 24).float().cuda(), rnd(7, c.t, 24).float().cuda()
    want = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=5)
    for t, v in ((dy, float("nan")), (c.x, float("inf")), (s, float("inf")), (u, float("nan"))):
        t[c.at[1]:c.at[2]] = v
    got = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=5)
    keep = torch.tensor([0, 2, 3, 4], device="cuda")
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep]) and not bool(a[1].isfinite().all())


def test_many_small_requests_among_many_rows():
    """More rows than are added one by one, in fewer places than requests have."""
    for lengths in ([1, 2, 3] * 60, [1] * 129, [7, 8] * 20 + [1] * 100):
        total = 6
        adapters = [i % (total + 1) - 1 for i in range(len(lengths))]
        for row in (False, True):
            Case(lengths, 200, 136, 20, adapters, total, "f16", row, gap=(3, 2), seed=len(lengths)).check("f32")


def test_streams_and_graphs():
    cases = [Case([1] * 20, 512, 512, 16, [i % 5 for i in range(20)], 5, seed=1), Case([400, 1, 90], 512, 512, 32, [2, 0, 1], 3, seed=2)]
    alone = [c.run("bf16") for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        both = [c.run("bf16", stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    c = cases[1]
    dy = rows16(rnd(3, c.t, 512), T["bf16"])

    def step():
        d, s = c.run("bf16")
        dx, u = mma.gemm_lora(dy, c.w, c.b, c.a, c.offsets, c.adapters, c.scales, b_layout="row", sums=True)
        return d, dx, *mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=3)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (5, 6):
        c.x.copy_(rnd(seed, *c.x.shape))
        c.offsets.copy_(ints([0, 100 + seed, 200, c.t]))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))


@pytest.mark.parametrize("lengths", [[1] * 1100 + [30], [1, 2] * 60])
def test_many_requests_captured_and_on_a_stream(lengths):
    """Rows in the order of their adapters: in a graph whose inputs change, and on a stream."""
    rng = random.Random(1)
    adapters = [rng.randint(-1, 5) for _ in lengths]
    c = Case(lengths, 136, 264, 48, adapters, 5, "bf16", seed=21)
    dy, u = rows16(rnd(5, c.t, 136), T["bf16"]), rnd(7, c.t, 48).float().cuda()

    def both():
        d, s = c.run("bf16")
        return d, s, *mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=5)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (31, 32):
        c.x.copy_(rnd(seed, c.t, 264).to(T["bf16"]))
        c.adapters.copy_(ints([rng.randint(-1, 5) for _ in lengths]))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d, s = c.run("bf16", stream=side)
    g = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=5, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (d, s, *g)))
