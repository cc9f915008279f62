"""Range of the norm's gradient: sums scaled by a power of two.

With eps = 0 the norm does not change when h is multiplied by 2^k, so its
gradient is divided by 2^k and the weights' is the same; every number in
between is scaled by a power of two, so the bits are those of k = 0 as long as
nothing over- or underflows.  1 / rms^3 by itself leaves FP32's range at some
2^42 either way.
"""
from __future__ import annotations

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [64, 1000, 4096, 20000])
@pytest.mark.parametrize("k", [-50, -45, 45, 50])
def test_scaled_rows(dtype, n, k):
    g = torch.Generator(device="cuda").manual_seed(n)
    dy, h = (torch.randn(9, n, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(dtype)
    want, want_w = mma.rmsnorm_backward(dy, h, w, eps=0.0)
    got, got_w = mma.rmsnorm_backward(dy, (h.float() * 2.0 ** k).to(dtype), w, eps=0.0)
    assert bool((got.float() == want.float() * 2.0 ** -k).all())
    assert bool((got_w == want_w).all())
