"""Products start beside the kernel before them (programmatic launch); their
bounded waits begin only when that kernel has ended, however long it takes.

The long one is a weight gradient of one tile over 7e8 rows of 16 bytes, on
two of the SMs: longer than the limit of two seconds of a wait.
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


def test_products_wait_for_a_long_kernel():
    tokens = 700_000_000
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB of device memory")
    x = torch.zeros(tokens, 8, dtype=torch.bfloat16, device="cuda")
    x[::1 << 22] = 1
    rows = float((tokens + (1 << 22) - 1) >> 22)
    at = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    a, sa = mma.quantize_f8(torch.randn(700, 512, device="cuda"))
    b, sb = mma.quantize_f8(torch.randn(384, 512, device="cuda"), block_rows=128)
    e = torch.randn(3, 384, 512, device="cuda").bfloat16()
    y = torch.randn(500, 512, device="cuda").bfloat16()
    off = torch.tensor([0, 70, 70, 500], dtype=torch.int32, device="cuda")

    later = [lambda: mma.gemm_f8(a[:1], sa[:1], b, sb), lambda: mma.gemm_f8(a, sa, b, sb),
             lambda: mma.gemm_grouped(y, e, off), lambda: mma.gemm_grouped_wgrad(y, y, off)]
    for call in later:
        want = call()
        torch.cuda.synchronize()
        t0 = time.time()
        dw = mma.gemm_grouped_wgrad(x, x, at)
        got = call()
        torch.cuda.synchronize()
        took = time.time() - t0
        binding.device_status()
        assert took > 2.2, took
        assert bool((dw == rows).all())
        assert bool((got == want).all())
