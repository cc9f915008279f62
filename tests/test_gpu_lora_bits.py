"""How many bits the rows' sums keep on their way through the products with adapters
and the adapters' gradients.

Tolerances.  With a 16-bit result the sums are two numbers of 16 bits, off by U^2 of
them (BF16 2^-16, FP16 2^-22) and 2^-38 of the largest; the products are off by SUM of
their magnitudes; the result is rounded once, by half a step.
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


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,r", [([300, 20, 1, 9], 64), ([5000], 16), ([700, 400], 128)])
def test_product_in_16_bits(lengths, r, kind, row):
    """The adapters' part alone: the shared matrix is zero."""
    c = Case(lengths, 520, 264, r, list(range(len(lengths))), len(lengths), kind, row, seed=r)
    c.w.zero_()
    got, _ = c.run(kind)
    want, mag, u_in, s64, _ = c.want()
    top = s64.abs().amax(1, keepdim=True) * host(c.b).abs().sum(1 if row else 2).max()
    tol = mag + u_in * U[kind] ** 2 + 2.0 ** -37 * top
    lim = (want.abs() + tol) * U[kind] + tol + STEP[kind]
    err = (host(got) - want).abs()
    assert bool((err <= lim).all()), float((err / lim).max())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,r", [([300], 64), ([100, 1, 40] * 3, 16), ([2000, 30], 128), ([1] * 200, 32)])
def test_gradients_in_16_bits(lengths, r, kind):
    total = 3
    c = Case(lengths, 264, 392, r, [i % total for i in range(len(lengths))], total, kind, seed=r)
    dy = rows16(rnd(5, c.t, 264), T[kind])
    s, u = rnd(6, c.t, r).float().cuda(), rnd(7, c.t, r).float().cuda()
    got = mma.gemm_lora_wgrad(dy, c.x, s, u, c.offsets, c.adapters, adapters_total=total, out_dtype=T[kind])
    a64, b64, ma, mb = wgrad_want(c, dy, s, u)
    for g, ref, mag in ((got[0], a64, ma), (got[1], b64, mb)):
        # (2^-38 of a column's largest sum is below 2^-34 of a row's magnitude)
        tol = mag * (SUM + U[kind] ** 2) + 2.0 ** -34 * mag.max()
        lim = (ref.abs() + tol) * U[kind] + tol + STEP[kind]
        err = (host(g) - ref).abs()
        assert bool((err <= lim).all()), float((err / lim).max())
