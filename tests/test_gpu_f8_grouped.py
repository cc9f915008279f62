"""Products of scaled 8-bit operands and products grouped by expert, against
the definitions in 64 bits.

Tolerance of a sum of K products with magnitudes |a||b| that add up to S.
One block (128 terms for 8-bit operands, 256 for 16-bit) is summed by the
tensor core, whose additions may each drop what lies below 2^-23 of the
running sum: at most 2^-15 S.  The blocks are added in FP32 to nearest, K / 128
additions and three more roundings for the scales: (K / 128 + 4) 2^-24 (S + |C|).
The result's own rounding is half an ulp of its type.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MAX = {"e4m3": 448.0, "e5m2": 57344.0}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(seed, *shape):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


def rows16(x, dtype=None, pad=0):
    """x with rows on 16-byte boundaries and NaN in the gaps."""
    dtype = dtype or x.dtype
    *lead, n = x.shape
    per = 16 // torch.empty((), dtype=dtype).element_size()
    big = torch.full((*lead, -(-n // per) * per + pad * per), float("nan"),
                     device="cuda").to(dtype)
    big.view(torch.uint8 if dtype.itemsize == 1 else dtype)[..., :n] = \
        x.to(dtype).view(torch.uint8) if dtype.itemsize == 1 else x.to(dtype)
    return big[..., :n]


def f8_operand(seed, m, k, f, rows, spread=1.0):
    """Random 8-bit values over the format's range and scales of all sizes."""
    q = rnd(seed, m, k)
    q = (q / q.abs().max() * MAX[f]).to(F8[f])
    s = torch.exp(spread * rnd(seed + 1, -(-m // rows), -(-k // 128))) / MAX[f]
    return rows16(q), s


def value(q, s, rows):
    m, k = q.shape
    return q.double() * s.double().repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :k]


def close(got, want, mag, k, what, block=2.0 ** -15):
    err = (got.double() - want).abs()
    bound = mag * (block + (k / 128 + 4) * 2.0 ** -24) + want.abs() * U[got.dtype] * (1 + 2.0 ** -8)
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {got.numel()} off, worst "
                                 f"{float((err / bound).nan_to_num(1e30).max()):.3g} bounds")


class Guard:
    """A (..., m, n) result inside canaries: a row above and below and `pad`
    columns beside it."""

    def __init__(self, m, n, dtype, pad=3, slices=1):
        self.big = torch.full((slices * (m + 2), n + pad), 123.0, device="cuda").to(dtype)
        self.m, self.n, self.slices = m, n, slices
        v = self.big.view(slices, m + 2, n + pad)[:, 1:-1, :n]
        self.view = v if slices > 1 else v[0]

    def check(self):
        b = self.big.view(self.slices, self.m + 2, -1).clone()
        b[:, 1:-1, :self.n] = 123.0
        assert bool((b == 123.0).all()), "written outside the result"


# ------------------------------------------------------------- 8-bit product

def run_f8(m, n, k, *, fa="e4m3", fb="e4m3", rows=128, d="bf16", c=False, inplace=False,
           order="block"):
    a, sa = f8_operand(1, m, k, fa, 1)
    b, sb = f8_operand(3, n, k, fb, rows)
    if order == "block":
        sa, sb = sa.t().contiguous().t(), sb.t().contiguous().t()
    dt = T[d]
    scale = (k ** 0.5)
    C = (scale * rnd(5, m, n)).to(dt) if c else None
    g = Guard(m, n, dt)
    if inplace:
        g.view.copy_(C)
        out = mma.gemm_f8(a, sa, b, sb, g.view, g.view)
    else:
        out = mma.gemm_f8(a, sa, b, sb, C, g.view)
    av, bv = value(a, sa, 1), value(b, sb, rows)
    want = av @ bv.t() + (C.double() if c else 0)
    mag = av.abs() @ bv.abs().t() + (C.double().abs() if c else 0)
    close(out, want, mag, k, f"{m}x{n}x{k}")
    g.check()


@pytest.mark.parametrize("m", [1, 3, 16, 17, 33, 64, 100, 129, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (128, 128), (130, 129), (520, 1000), (64, 16), (257, 4096)])
def test_f8_shapes(m, n, k):
    run_f8(m, n, k)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
def test_f8_types(fa, fb, d, rows):
    run_f8(200, 264, 700, fa=fa, fb=fb, d=d, rows=rows, c=True)
    run_f8(9, 264, 700, fa=fa, fb=fb, d=d, rows=rows)


@pytest.mark.parametrize("m", [5, 260, 1500])
def test_f8_scale_strides_and_in_place(m):
    run_f8(m, 640, 1280, order="row", d="f32")
    run_f8(m, 640, 1280, rows=1, order="row", d="bf16", c=True)
    run_f8(m, 641, 1280, d="f32", c=True, inplace=True)


@pytest.mark.parametrize("m,n,k", [(300, 520, 1000), (1300, 264, 512), (257, 1032, 130)])
@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,c", [(128, False), (128, True), (1, False)])
def test_f8_aligned_results(m, n, k, d, rows, c):
    """Results whose rows start on 16-byte boundaries take the wide stores."""
    a, sa = f8_operand(1, m, k, "e4m3", 1)
    b, sb = f8_operand(3, n, k, "e4m3", rows)
    C = rnd(5, m, n + 8).to(T[d])[:, :n] if c else None
    g = Guard(m, n, T[d], pad=8)
    mma.gemm_f8(a, sa, b, sb, C, g.view)
    av, bv = value(a, sa, 1), value(b, sb, rows)
    add = C.double() if c else 0
    close(g.view, av @ bv.t() + add, av.abs() @ bv.abs().t() + (add.abs() if c else 0), k, "aligned")
    g.check()


def test_chained_calls_wait_for_each_other():
    """Calls start before the ones before them have ended: a chain without
    synchronisation has the bits of one with."""
    k = 1024
    w = [mma.quantize_f8(rnd(20 + i, k, k) / k ** 0.5, block_rows=128) for i in range(3)]
    e = rnd(30, 3, k, k).to(torch.bfloat16) / 32

    def chain(rows, sync):
        at = off([0, rows // 3, rows // 3, rows])
        x, out = rnd(31, rows, k).to(torch.bfloat16), []
        for i in range(12):
            q, s = mma.quantize_f8(x)
            y = mma.gemm_f8(q, s, *w[i % 3])
            sync()
            z = mma.gemm_grouped(y, e, at)
            sync()
            z = mma.gemm_grouped(z, e, at, b_layout="row", D=y)   # over its own input's input
            sync()
            out.append(mma.gemm_grouped_wgrad(z, y, at, out_dtype=torch.bfloat16))
            sync()
            x = (z / z.float().abs().mean()).to(torch.bfloat16)
        return x, out

    for rows in (5, 40, 700):
        want, want_w = chain(rows, torch.cuda.synchronize)
        got, got_w = chain(rows, lambda: None)
        assert bool((got == want).all())
        assert all(bool((a == b).all()) for a, b in zip(got_w, want_w))


def test_f8_many_tiles():
    run_f8(2300, 2200, 512)
    run_f8(2300, 2200, 640, rows=1, d="f32")


@pytest.mark.parametrize("m,n,k", [(3001, 901, 300), (130, 20000, 136), (5000, 520, 129),
                                   (20500, 1, 260), (257, 10240, 16)])
@pytest.mark.parametrize("d,c", [("bf16", True), ("f16", False), ("f32", True), ("f32", False)])
def test_f8_row_scales_many_tiles(m, n, k, d, c):
    """More 128 x 128 tiles than SMs: pairs of CTAs."""
    run_f8(m, n, k, rows=1, d=d, c=c)
    run_f8(m, n, k, rows=1, d=d, c=True, inplace=True, order="row")


@pytest.mark.parametrize("m,n", [(300, 520), (129, 1), (700, 1000)])
@pytest.mark.parametrize("rows", [1, 128])
def test_f8_few_tiles_long_reduction(m, n, rows):
    run_f8(m, n, 4200, rows=rows, c=True)
    run_f8(m, n, 4096, rows=rows, d="f32")


def test_f8_empty_reduction():
    a, sa = torch.empty(7, 0, device="cuda").to(F8["e4m3"]), torch.empty(7, 0, device="cuda")
    b, sb = torch.empty(300, 0, device="cuda").to(F8["e4m3"]), torch.empty(3, 0, device="cuda")
    assert bool((mma.gemm_f8(a, sa, b, sb) == 0).all())
    c = rnd(1, 7, 300).to(torch.bfloat16)
    assert bool((mma.gemm_f8(a, sa, b, sb, c) == c).all())
    assert mma.gemm_f8(a[:0], sa[:0], b, sb).shape == (0, 300)


def test_f8_specials_stay_in_their_row():
    """NaN values and infinite scales reach their own row or column only."""
    m, n, k = 140, 300, 512
    a, sa = f8_operand(1, m, k, "e4m3", 1)
    b, sb = f8_operand(3, n, k, "e4m3", 128)
    base = mma.gemm_f8(a, sa, b, sb, out_dtype=torch.float32)
    a.view(torch.uint8)[5, 200] = 0x7F
    sa[77, 1] = float("inf")
    b.view(torch.uint8)[44, 511] = 0xFF
    out = mma.gemm_f8(a, sa, b, sb, out_dtype=torch.float32)
    assert bool(torch.isnan(out[5]).all()) and bool(torch.isnan(out[:, 44]).all())
    assert not bool(torch.isfinite(out[77]).any())
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    keep[5] = keep[77] = False
    keep[:, 44] = False
    assert bool((out[keep] == base[keep]).all())


def test_f8_chain_from_the_quantisers():
    """Norm, product, and the product's two gradients on quantised operands:
    each against the same formula on the quantised values in 64 bits."""
    m, n, k = 300, 384, 640
    x, r = rnd(1, m, k).to(torch.bfloat16), rnd(2, m, k).to(torch.bfloat16)
    q, s, _ = mma.rmsnorm_f8(x, torch.ones(k, dtype=torch.bfloat16, device="cuda"), r)
    w = rnd(3, n, k) / k ** 0.5
    wq, ws = mma.quantize_f8(w, block_rows=128)
    y = mma.gemm_f8(q, s, wq, ws)
    qv, wv = value(q, s, 1), value(wq, ws, 128)
    close(y, qv @ wv.t(), qv.abs() @ wv.abs().t(), k, "forward")
    dy = rnd(4, m, n).to(torch.bfloat16)
    dq, ds = mma.quantize_f8(dy, fmt="e5m2")
    wt, wts = mma.quantize_f8(w, block_rows=128, transpose=True)
    assert bool((wt.t().float() == wq.float()).all()) and bool((wts.t() == ws).all())
    dx = mma.gemm_f8(dq, ds, wt, wts)
    dv = value(dq, ds, 1)
    close(dx, dv @ wv, dv.abs() @ wv.abs(), n, "input gradient")
    dt, dts = mma.quantize_f8(dy, fmt="e5m2", transpose=True)
    xt, xts = mma.quantize_f8(rnd(5, m, k).to(torch.bfloat16), transpose=True)
    dw = mma.gemm_f8(dt, dts, xt, xts, out_dtype=torch.float32)
    av, bv = value(dt, dts, 1), value(xt, xts, 1)
    close(dw, av @ bv.t(), av.abs() @ bv.abs().t(), m, "weight gradient")


# ------------------------------------------------------------------ grouped

OFFSETS = {
    "even": [0, 100, 200, 300, 400],
    "ragged": [0, 1, 1, 130, 131, 400],
    "empty ends": [0, 0, 37, 400, 400, 400],
    "gaps": [3, 20, 20, 389],           # rows before and behind belong to nobody
    "one": [0, 400],
    "none": [0, 0, 0],
    "tiny": [0] + list(range(1, 41)) + [400],
}


def off(at):
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def grouped64(a, b, at, row):
    out = torch.zeros(a.shape[0], b.shape[2 if row else 1], dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        w = b[e].double()
        out[lo:hi] = a[lo:hi].double() @ (w if row else w.t())
    return out


@pytest.mark.parametrize("at", list(OFFSETS))
@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("t,d", [("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
def test_grouped(at, layout, t, d):
    at = OFFSETS[at]
    tokens, n, k = 400, 200, 328
    row = layout == "row"
    a = rows16(rnd(1, tokens, k), T[t], 1)
    e = len(at) - 1
    b = rows16(rnd(2, e, *((k, n) if row else (n, k))), T[t], 1)
    c = rnd(3, tokens, n).to(T[d])
    g = Guard(tokens, n, T[d])
    for C in (None, c):
        g.view.fill_(55.0)
        mma.gemm_grouped(a, b, off(at), C, g.view, b_layout=layout)
        want = grouped64(a, b, at, row) + (0 if C is None else C.double())
        mag = grouped64(a.abs(), b.abs(), at, row) + (0 if C is None else C.double().abs())
        lo, hi = at[0], at[-1]
        close(g.view[lo:hi], want[lo:hi], mag[lo:hi], k, "grouped")
        assert bool((g.view[:lo] == 55).all()) and bool((g.view[hi:] == 55).all())
        g.check()


@pytest.mark.parametrize("tokens,e,n,k", [(1, 1, 1, 1), (1, 8, 130, 64), (7, 3, 64, 1000),
                                          (64, 64, 256, 512), (2000, 3, 1000, 72), (3000, 5, 300, 2048)])
@pytest.mark.parametrize("layout", ["col", "row"])
def test_grouped_shapes(tokens, e, n, k, layout):
    g = torch.Generator().manual_seed(7)
    at = sorted(int(v) for v in torch.randint(0, tokens + 1, (e - 1,), generator=g))
    at = [0] + at + [tokens]
    row = layout == "row"
    a = rows16(rnd(1, tokens, k), torch.bfloat16)
    b = rows16(rnd(2, e, *((k, n) if row else (n, k))), torch.bfloat16)
    out = mma.gemm_grouped(a, b, off(at), b_layout=layout, out_dtype=torch.float32)
    close(out, grouped64(a, b, at, row), grouped64(a.abs(), b.abs(), at, row), k, "grouped")


def test_grouped_offsets_out_of_range():
    """Offsets that decrease or leave [0, T] are clamped; nothing outside the
    result is written."""
    a, b = rnd(1, 50, 64).to(torch.bfloat16), rnd(2, 4, 72, 64).to(torch.bfloat16)
    g = Guard(50, 72, torch.bfloat16)
    mma.gemm_grouped(a, b, off([-9, 20, 10, 1 << 30, 7]), None, g.view)
    at = [0, 20, 20, 50, 50]
    close(g.view, grouped64(a, b, at, False), grouped64(a.abs(), b.abs(), at, False), 64, "clamped")
    g.check()
    dw = mma.gemm_grouped_wgrad(rnd(3, 50, 72).to(torch.bfloat16), a, off([-9, 20, 10, 1 << 30, 7]))
    assert bool((dw[1] == 0).all()) and bool((dw[3] == 0).all()) and bool(torch.isfinite(dw).all())


def test_grouped_other_groups_do_not_leak():
    """NaN and infinity in one group's rows or weights stay in that group."""
    at, k, n = [0, 33, 90, 200], 128, 160
    a, b = rnd(1, 200, k).to(torch.bfloat16), rnd(2, 3, n, k).to(torch.bfloat16)
    base = mma.gemm_grouped(a, b, off(at))
    dy = rnd(3, 200, n).to(torch.bfloat16)
    base_w = mma.gemm_grouped_wgrad(dy, a, off(at))
    a2, b2, dy2 = a.clone(), b.clone(), dy.clone()
    a2[33:90] = float("nan")
    dy2[33:90] = float("inf")
    b2[1] = float("inf")
    out = mma.gemm_grouped(a2, b2, off(at))
    keep = list(range(33)) + list(range(90, 200))
    assert bool((out[keep] == base[keep]).all()) and bool(torch.isnan(out[33:90]).all())
    dw = mma.gemm_grouped_wgrad(dy2, a2, off(at))
    assert bool((dw[0] == base_w[0]).all()) and bool((dw[2] == base_w[2]).all())
    assert bool(torch.isnan(dw[1]).all())


def wgrad64(dy, x, at):
    return torch.stack([dy[lo:hi].double().t() @ x[lo:hi].double() for lo, hi in zip(at, at[1:])])


@pytest.mark.parametrize("at", list(OFFSETS))
@pytest.mark.parametrize("t,d", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_grouped_wgrad(at, t, d):
    at = OFFSETS[at]
    tokens, n, k, e = 400, 200, 328, len(OFFSETS) and len(at) - 1
    dy, x = rows16(rnd(1, tokens, n), T[t], 1), rows16(rnd(2, tokens, k), T[t])
    want, mag = wgrad64(dy, x, at), wgrad64(dy.abs(), x.abs(), at)
    g = Guard(n, k, T[d], slices=e)
    D = g.view if e > 1 else g.view[None]
    mma.gemm_grouped_wgrad(dy, x, off(at), None, D)
    close(D, want, mag, tokens, "wgrad")
    g.check()
    c = rnd(3, e, n, k).to(T[d])
    D.copy_(c)
    mma.gemm_grouped_wgrad(dy, x, off(at), D, D)   # accumulation
    close(D, want + c.double(), mag + c.double().abs(), tokens, "wgrad + C")
    g.check()


@pytest.mark.parametrize("tokens,e,n,k", [(1, 1, 8, 8), (1, 2, 1, 1), (65, 2, 264, 136), (5000, 3, 700, 520),
                                          (300, 40, 257, 129)])
def test_grouped_wgrad_shapes(tokens, e, n, k):
    g = torch.Generator().manual_seed(9)
    at = [0] + sorted(int(v) for v in torch.randint(0, tokens + 1, (e - 1,), generator=g)) + [tokens]
    dy, x = rows16(rnd(1, tokens, n), torch.bfloat16), rows16(rnd(2, tokens, k), torch.bfloat16)
    out = mma.gemm_grouped_wgrad(dy, x, off(at))
    close(out, wgrad64(dy, x, at), wgrad64(dy.abs(), x.abs(), at), tokens, "wgrad")


def test_grouped_wgrad_without_rows():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    out = mma.gemm_grouped_wgrad(z, z, off([0, 0, 0]))
    assert out.shape == (2, 64, 64) and bool((out == 0).all())
    c = rnd(1, 2, 64, 64)
    assert bool((mma.gemm_grouped_wgrad(z, z, off([0, 0, 0]), c) == c).all())
    assert mma.gemm_grouped(z, rnd(2, 2, 32, 64).to(torch.bfloat16), off([0, 0, 0])).shape == (0, 32)


def test_grouped_gradients_against_differences():
    """<G, D> is linear in A and in B, so its difference quotient along a
    direction is the inner product of that direction with the gradient; both
    in the type's exact values, the tolerance that of the products."""
    at, n, k = [0, 40, 40, 111], 96, 80
    a, b = rnd(1, 111, k).to(torch.bfloat16), rnd(2, 3, n, k).to(torch.bfloat16)
    g = rnd(3, 111, n).to(torch.bfloat16)
    da = mma.gemm_grouped(g, b, off(at), b_layout="row", out_dtype=torch.float32)
    db = mma.gemm_grouped_wgrad(g, a, off(at))
    va, vb = rnd(4, 111, k).double(), rnd(5, 3, n, k).double()
    step = 1e-3
    f = lambda x, w: float((g.double() * grouped64(x, w, at, False)).sum())  # noqa: E731
    qa = (f(a.double() + step * va, b) - f(a.double() - step * va, b)) / (2 * step)
    qb = (f(a, b.double() + step * vb) - f(a, b.double() - step * vb)) / (2 * step)
    mag_a = float((grouped64(g.abs(), b.abs(), at, True) * va.abs()).sum())
    mag_b = float((wgrad64(g.abs(), a.abs(), at) * vb.abs()).sum())
    assert abs(qa - float((da.double() * va).sum())) <= 2.0 ** -15 * mag_a
    assert abs(qb - float((db.double() * vb).sum())) <= 2.0 ** -15 * mag_b


@pytest.mark.parametrize("at", list(OFFSETS))
@pytest.mark.parametrize("rows", [1, 128])
def test_grouped_f8(at, rows):
    at = OFFSETS[at]
    tokens, n, k, e = 400, 200, 400, len(at) - 1
    a, sa = f8_operand(1, tokens, k, "e4m3", 1)
    ops = [f8_operand(10 + 2 * i, n, k, "e4m3", rows) for i in range(e)]
    b = rows16(torch.stack([q.view(torch.uint8) for q, _ in ops]).view(F8["e4m3"]))
    sb = torch.stack([s for _, s in ops])
    bv = torch.stack([value(q, s, rows) for q, s in ops])
    av = value(a, sa, 1)
    g = Guard(tokens, n, torch.bfloat16)
    g.view.fill_(55.0)
    mma.gemm_grouped_f8(a, sa.t().contiguous().t(), b, sb, off(at), None, g.view)
    lo, hi = at[0], at[-1]
    close(g.view[lo:hi], grouped64(av, bv, at, False)[lo:hi],
          grouped64(av.abs(), bv.abs(), at, False)[lo:hi], k, "grouped f8")
    assert bool((g.view[:lo] == 55).all()) and bool((g.view[hi:] == 55).all())
    g.check()


@pytest.mark.parametrize("tokens,e", [(1, 4), (20, 16), (3000, 4)])
def test_grouped_f8_shapes(tokens, e):
    n, k = 520, 1100
    g = torch.Generator().manual_seed(3)
    at = [0] + sorted(int(v) for v in torch.randint(0, tokens + 1, (e - 1,), generator=g)) + [tokens]
    a, sa = f8_operand(1, tokens, k, "e4m3", 1)
    ops = [f8_operand(10 + 2 * i, n, k, "e4m3", 128) for i in range(e)]
    b = rows16(torch.stack([q.view(torch.uint8) for q, _ in ops]).view(F8["e4m3"]))
    sb = torch.stack([s for _, s in ops])
    bv, av = torch.stack([value(q, s, 128) for q, s in ops]), value(a, sa, 1)
    out = mma.gemm_grouped_f8(a, sa, b, sb, off(at), out_dtype=torch.float32)
    close(out, grouped64(av, bv, at, False), grouped64(av.abs(), bv.abs(), at, False), k, "f8")


@pytest.mark.parametrize("rows", [1, 128])
def test_grouped_f8_many_rows(rows):
    at = [3, 3, 700, 1213, 1214, 2900]
    tokens, n, k, e = 3000, 1301, 400, 5
    a, sa = f8_operand(1, tokens, k, "e4m3", 1)
    ops = [f8_operand(10 + 2 * i, n, k, "e4m3", rows) for i in range(e)]
    b = rows16(torch.stack([q.view(torch.uint8) for q, _ in ops]).view(F8["e4m3"]))
    sb = torch.stack([s for _, s in ops])
    bv, av = torch.stack([value(q, s, rows) for q, s in ops]), value(a, sa, 1)
    c = rnd(9, tokens, n).to(torch.bfloat16)
    g = Guard(tokens, n, torch.bfloat16)
    g.view.fill_(55.0)
    mma.gemm_grouped_f8(a, sa, b, sb, off(at), c, g.view)
    want = grouped64(av, bv, at, False) + c.double()
    mag = grouped64(av.abs(), bv.abs(), at, False) + c.double().abs()
    lo, hi = at[0], at[-1]
    close(g.view[lo:hi], want[lo:hi], mag[lo:hi], k, "f8")
    assert bool((g.view[:lo] == 55).all()) and bool((g.view[hi:] == 55).all())
    g.check()


def test_repeatable_other_stream_and_graph():
    at = off([0, 70, 70, 500])
    a, b = rnd(1, 500, 256).to(torch.bfloat16), rnd(2, 3, 384, 256).to(torch.bfloat16)
    qa, sa = mma.quantize_f8(a)
    qb, sb = mma.quantize_f8(b.view(-1, 256), block_rows=128)
    qb, sb = qb.view(3, 384, 256), sb.t().contiguous().t().contiguous().view(3, 3, 2)

    def both():
        return (mma.gemm_grouped(a, b, at), mma.gemm_grouped_f8(qa, sa, qb, sb, at),
                mma.gemm_grouped_wgrad(b[0].t().contiguous()[:256], a[:256], at.clamp(max=256)),
                mma.gemm_f8(qa, sa, qb[0], sb[0]))

    first = both()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        second = both()
    other.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(first, second, third):
        assert bool((x == y).all()) and bool((x == z).all())


def test_operands_beyond_32_bit_offsets():
    """More than 2^31 elements of weights, and of the result."""
    e, n, k = 36, 8192, 8192
    b = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
    b[-1] = rnd(1, n, k)
    a = rnd(2, 5, k).to(torch.bfloat16)
    at = [0] * e + [5]
    out = mma.gemm_grouped(a, b, off(at), out_dtype=torch.float32)
    want, mag = a.double() @ b[-1].double().t(), a.double().abs() @ b[-1].double().abs().t()
    close(out, want, mag, k, "far expert")
    del b, want, mag
    tokens, n, k = 275_000, 8192, 64
    a = torch.zeros(tokens, k, dtype=torch.bfloat16, device="cuda")
    a[-300:] = rnd(3, 300, k)
    b = rnd(4, 2, n, k).to(torch.bfloat16)
    out = mma.gemm_grouped(a, b, off([0, 1000, tokens]))
    close(out[-300:], a[-300:].double() @ b[1].double().t(),
          a[-300:].double().abs() @ b[1].double().abs().t(), k, "far rows")
    assert bool((out[:-300] == 0).all())
