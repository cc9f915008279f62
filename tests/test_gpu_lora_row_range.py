"""Products with adapters of FP16 matrices whose rows' sums are far smaller or larger
than FP16's numbers.

Tolerances.  The sums enter a product as numbers of 16 bits, scaled by a power of two
for each row that brings the largest to 2^13 or
above: one number is off by half a step, 2^-11, two by 2^-22 of the sum, and by
2^-25 (half of FP16's smallest step) of 2^13, so 2^-38 of the largest.  The products
themselves are off by SUM of their magnitudes, as in the other tests of adapters.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from mixed_precision_dense_02_gb300 import binding
from test_gpu_lora import STEP, U, Case, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("lengths", [[200, 9, 30, 1, 100], [8] * 40, [4000, 300]])
@pytest.mark.parametrize("out,size,b_size", [("f32", 1e-7, 1.0), ("f32", 1e7, 1.0), ("f32", 1e-25, 1.0), ("f16", 1e6, 2.0 ** -12)])
def test_products_of_small_and_large_sums(lengths, row, out, size, b_size):
    """Adapters alone (the shared matrix is zero), whose scales differ from one to the next."""
    total = 4
    c = Case(lengths, 264, 136, 40, [i % total for i in range(len(lengths))], total, "f16", row, gap=(1, 3), seed=7)
    c.w.zero_()
    c.b *= b_size
    c.scales *= size * torch.tensor([1.0, 0.01, 0.3, 1e-3], device="cuda")
    got, s = c.run(out)
    want, mag, u_in, s64, s_tol = c.want()
    assert bool(((host(s) - s64).abs() <= s_tol + 2.0 ** -23 * s64.abs()).all())
    b = host(c.b).transpose(1, 2) if row else host(c.b)
    top = torch.zeros(c.t, 264, dtype=torch.float64)
    for j, (i0, i1) in enumerate(zip(c.at, c.at[1:])):
        top[i0:i1] = s64[i0:i1].abs().amax(1, keepdim=True) * b[c.who(j)].abs().sum(1)[None]
    # (the sums' own error is 2^-38 of the largest too, and less)
    tol = mag + u_in * (2.0 ** -22 if out == "f32" else U["f16"]) + 2.0 ** -37 * top
    lim = (want.abs() + tol) * U[out] + tol + STEP[out]
    err = (host(got) - want).abs()
    assert bool((err <= lim).all()), float((err / lim).max())


def test_bad_sums_stay_in_their_row():
    """One row's sums are infinite, its neighbours' in the same request are not."""
    c = Case([150, 30], 136, 200, 16, [0, 1], 2, "f16", seed=5)
    clean, _ = c.run("f32")
    c.x[40, 7] = float("inf")
    got, _ = c.run("f32")
    assert not bool(got[40].isfinite().any())
    got[40] = clean[40]
    assert torch.equal(got, clean)
