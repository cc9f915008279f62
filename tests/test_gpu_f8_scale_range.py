"""Products over the range of scales: both scales multiplied by powers of two
whose product stays in FP32's range give the same bits, multiplied by it."""
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


@pytest.mark.parametrize("m", [1, 100, 1500])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("ka,kb", [(-50, -49), (-110, 60), (60, -110), (40, 40), (80, -80)])
def test_scales(m, rows, ka, kb):
    g = torch.Generator(device="cuda").manual_seed(m)
    a, sa = mma.quantize_f8(torch.randn(m, 640, generator=g, device="cuda"))
    b, sb = mma.quantize_f8(torch.randn(1300, 640, generator=g, device="cuda"), block_rows=rows)
    want = mma.gemm_f8(a, sa, b, sb, out_dtype=torch.float32)
    got = mma.gemm_f8(a, sa * 2.0 ** ka, b, sb * 2.0 ** kb, out_dtype=torch.float32)
    assert bool((got == want * 2.0 ** (ka + kb)).all())
