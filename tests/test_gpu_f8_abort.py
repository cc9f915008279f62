"""The kernels of the norm, the quantiser and the products, when a wait runs out:
they store nothing, end by themselves and leave the context usable."""
from __future__ import annotations

import time

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

MMA_OK, MMA_ERR_TIMEOUT = 0, 5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_nothing_is_stored_after_a_failed_wait(kernel):
    stream = torch.cuda.current_stream().cuda_stream
    assert binding.mma_device_status(stream) == MMA_OK
    x = torch.randn(1024, 1024, device="cuda").bfloat16()
    out = torch.full((1024, 1024), 0x5A5A, dtype=torch.int16, device="cuda")
    s = torch.full((8192,), -7.0, device="cuda")
    ws = torch.zeros(456 * 1024, device="cuda") if kernel == 2 else None
    for _ in range(2):
        t0 = time.time()
        assert binding.mma_selftest_f8_abort(kernel, 20_000_000, x.data_ptr(), out.data_ptr(), s.data_ptr(),
                                             None if ws is None else ws.data_ptr(), stream) == MMA_OK
        torch.cuda.synchronize()
        assert 0.01 < time.time() - t0 < 10.0
        assert binding.mma_device_status(stream) == MMA_ERR_TIMEOUT
        assert binding.mma_device_status(stream) == MMA_OK
    assert bool((out == 0x5A5A).all())
    if kernel == 2:
        assert bool((ws == 0).all()) and bool((s[:1024] == 0).all()) and bool((s[1024:] == -7).all())
        dx, _ = mma.rmsnorm_backward(x, x, x[0])
        assert bool(torch.isfinite(dx.float()).all())
    else:
        assert bool((s == -7).all())
        q, sc = mma.quantize_f8(x, block_rows=128 if kernel == 0 else 1, transpose=kernel == 1)
        v = q.float() * sc.repeat_interleave(128 if kernel == 0 else 1, 0).repeat_interleave(128, 1)
        want = (x.t() if kernel == 1 else x).float()
        assert bool(((v - want).abs() <= want.abs() / 16 + sc.max() / 1024).all())
    assert binding.mma_device_status(stream) == MMA_OK


@pytest.mark.parametrize("kernel", [3, 4, 5])
def test_products_end_after_a_failed_wait(kernel):
    """A cluster that shares the k range, pairs with row scales of A, and the
    ragged reduction; each wait takes its own two seconds."""
    stream = torch.cuda.current_stream().cuda_stream
    assert binding.mma_device_status(stream) == MMA_OK
    x = torch.zeros(1024, 1024, dtype=torch.int16, device="cuda")
    out = torch.full((1024, 1024), 0x5A5A, dtype=torch.int16, device="cuda")
    s = torch.zeros(8192, dtype=torch.int32, device="cuda")
    s[1] = 1000  # (as offsets: one group that ends inside a step of 16)
    t0 = time.time()
    assert binding.mma_selftest_f8_abort(kernel, 20_000_000, x.data_ptr(), out.data_ptr(), s.data_ptr(), None,
                                         stream) == MMA_OK
    torch.cuda.synchronize()
    assert 1.5 < time.time() - t0 < 30.0
    assert binding.mma_device_status(stream) == MMA_ERR_TIMEOUT
    assert binding.mma_device_status(stream) == MMA_OK
    assert bool((out == 0x5A5A).all())
    # and the same shapes again, right
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(1024, 1024, generator=g, device="cuda").bfloat16()
    if kernel == 5:
        got = mma.gemm_grouped_wgrad(w, w, s[:2], out_dtype=torch.float32)[0]
        a = b = w[:1000].double().t()
        bound = 2.0 ** -14
    else:
        q, sa = mma.quantize_f8(w[:1 if kernel == 3 else 1024])
        p, sb = mma.quantize_f8(w, block_rows=128)
        got = mma.gemm_f8(q, sa, p, sb, out_dtype=torch.float32)
        a = q.double() * sa.double().repeat_interleave(128, 1)
        b = p.double() * sb.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        bound = 2.0 ** -14
    assert bool(((got.double() - a @ b.t()).abs() <= bound * (a.abs() @ b.abs().t())).all())
    assert binding.mma_device_status(stream) == MMA_OK
