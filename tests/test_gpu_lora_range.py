"""Gradients of FP16 adapters from rows' sums that are far smaller or larger than FP16's
numbers.

Tolerances.  The sums enter a product as numbers of 16 bits, scaled by a power of two
for each column of at most 64 rows that brings the largest to 2^13 or
above: one number is off by half a step, 2^-11, two by 2^-22 of the sum, and by
2^-25 (half of FP16's smallest step) of 2^13, so 2^-38 of the largest.  The products
themselves are off by SUM of their magnitudes, as in the other tests of adapters.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding
from test_gpu_lora import STEP, SUM, T, U, Case, host, rnd, rows16, wgrad_want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def largest(c, low, m):
    """Per adapter, sum and feature: the largest sum times the features' magnitudes."""
    out = torch.zeros(c.total, low.shape[1], m.shape[1], dtype=torch.float64)
    for j, (i0, i1) in enumerate(zip(c.at, c.at[1:])):
        q = c.who(j)
        if q >= 0 and i1 > i0:
            out[q] += low[i0:i1].abs().amax(0)[:, None] * m[i0:i1].abs().sum(0)[None]
    return out


def check_wgrad(c, dy, s, u, out="f32"):
    got = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=c.total, out_dtype=T[out])
    a64, b64, ma, mb = wgrad_want(c, dy, s, u)
    rel = SUM + (2.0 ** -22 if out == "f32" else U["f16"])
    da_max = largest(c, host(u), host(c.x))
    db_max = largest(c, host(s), host(dy)).transpose(1, 2)
    for g, ref, mag, top in ((got[0], a64, ma, da_max), (got[1], b64, mb, db_max)):
        tol = mag * rel + 2.0 ** -38 * top
        lim = (ref.abs() + tol) * U[out] + tol + STEP[out]
        err = (host(g) - ref).abs()
        if out == "f16":  # numbers of 65520 and more are rounded to infinity
            err = torch.where((host(g) == ref.sign() * float("inf")) & (ref.abs() + lim >= 65520.0), 0.0, err)
        assert bool((err <= lim).all()), float((err / lim).max())
    return got


LENGTHS = [[300, 1, 70, 0, 5], [1] * 130 + [40], [64, 64, 65], [2, 1] * 90]


@pytest.mark.parametrize("out,s_size,u_size,m_size", [
    ("f32", 1e-6, 1e-7, 1.0), ("f32", 1e5, 1e6, 1.0), ("f32", 1.0, 1e-9, 1.0), ("f32", 1e-30, 1e30, 1.0),
    ("f32", 1e-4, 1e-5, 1.0), ("f16", 1e-6, 1e-7, 256.0), ("f16", 1e5, 1e6, 2.0 ** -9)])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("r", [16, 40, 128])
def test_gradients_of_small_and_large_sums(lengths, r, out, s_size, u_size, m_size):
    total = 5
    c = Case(lengths, 136, 200, r, [i % total for i in range(len(lengths))], total, "f16", gap=(3, 2), seed=r)
    c.x *= m_size
    dy = rows16(m_size * rnd(5, c.t, 136), T["f16"], 1)
    s, u = (s_size * rnd(6, c.t, r)).float().cuda(), (u_size * rnd(7, c.t, r)).float().cuda()
    check_wgrad(c, dy, s, u, out)


@pytest.mark.parametrize("sizes", [[1.0, 1e-9, 1e7], [1e-12, 3e4, 1e-3]])
def test_gradients_of_adapters_of_different_size(sizes):
    """Neighbours inside a block of rows, and the sums of one adapter of different size."""
    lengths = [30, 20, 50, 7, 100, 1, 200]
    c = Case(lengths, 136, 264, 24, [0, 1, 2, 1, 0, 2, 1], 3, "f16", seed=3)
    dy = rows16(rnd(5, c.t, 136), T["f16"])
    s, u = rnd(6, c.t, 24), rnd(7, c.t, 24)
    for j, (i0, i1) in enumerate(zip(c.at, c.at[1:])):
        s[i0:i1] *= sizes[c.who(j)]
        u[i0:i1] *= sizes[(c.who(j) + 1) % 3]
    check_wgrad(c, dy, s.float().cuda(), u.float().cuda())
    columns = 10.0 ** torch.linspace(-12, 8, 24, dtype=torch.float64)
    check_wgrad(c, dy, (s * columns).float().cuda(), (u * columns.flip(0)).float().cuda())
    rows = 10.0 ** (-8 * torch.rand(c.t, 1, generator=torch.Generator().manual_seed(1), dtype=torch.float64))
    check_wgrad(c, dy, (s * rows).float().cuda(), (u * rows).float().cuda())


def test_bad_sums_stay_in_their_column():
    c = Case([100, 90], 136, 200, 16, [0, 1], 2, "f16", seed=8)
    dy = rows16(rnd(5, c.t, 136), T["f16"])
    s, u = (1e-6 * rnd(6, c.t, 16)).float().cuda(), (1e6 * rnd(7, c.t, 16)).float().cuda()
    da, db = check_wgrad(c, dy, s, u)
    s[20, 3], u[150, 5] = float("inf"), float("nan")
    ga, gb = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=2)
    assert not bool(gb[0, :, 3].isfinite().any()) and bool(ga[1, 5].isnan().all())
    gb[0, :, 3], ga[1, 5] = db[0, :, 3], da[1, 5]
    assert torch.equal(ga, da) and torch.equal(gb, db)


def test_captured_and_replayed():
    """Sums of another size in each replay, their scales with them."""
    for lengths in ([200, 1, 90], [1, 2] * 90):
        c = Case(lengths, 136, 200, 32, [i % 3 for i in range(len(lengths))], 3, "f16", seed=4)
        dy = rows16(rnd(5, c.t, 136), T["f16"])

        def step():
            d, s = c.run("f32")
            dx, u = mma.gemm_lora(dy, c.w, c.b, c.a, c.offsets, c.adapters, c.scales, b_layout="row", sums=True)
            return d, s, dx, u, *mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=3)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for size in (1e-8, 1e6, 1.0):
            c.scales.copy_(size * torch.tensor([1.0, 0.01, 30.0]))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, step())), size
            check_wgrad(c, dy, out[1], out[3])
