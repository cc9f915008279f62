"""The shared product of adapters starts beside the kernel of the rows' sums; its bounded
waits are over before that kernel's end is waited for, however long it takes.

The long one: what one request of 16 rows adds to 2^26 columns, row-major, which one block
makes.  That is longer than the limit of two seconds of a wait.
"""
from __future__ import annotations

import time

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def test_a_long_kernel_of_sums():
    rows, n, k, r = 16, 1 << 26, 8, 128
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
    w = torch.empty(k, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    a = torch.randn(1, k, r, generator=g, device="cuda").bfloat16()
    b = torch.empty(1, r, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    at = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    d, s = mma.gemm_lora(x, w, a, b, at, b_layout="row", sums=True)
    torch.cuda.synchronize()
    took = time.time() - t0
    binding.device_status()
    assert took > 2.2, took
    # a tensor core's sums and those of 128 FP32 products: 2^-16 of the magnitudes
    for i in (0, n // 3 // 8 * 8, n - 5000):
        c = slice(i, i + 5000)
        low = x.double() @ a[0].double()
        want = x.double() @ w[:, c].double() + low @ b[0, :, c].double()
        mag = x.double().abs() @ w[:, c].double().abs() + (x.double().abs() @ a[0].double().abs()) @ b[0, :, c].double().abs()
        tol = 2.0 ** -16 * mag
        assert bool(((d[:, c].double() - want).abs() <= (want.abs() + tol) * 2.0 ** -8 + tol).all())
