"""What follows an adapters' gradient that adds nothing: its workspace is free for the
work after it, also for a kernel that starts beside the one before."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding
from test_gpu_lora import T, ints, rnd, rows16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_nothing_to_add(kind):
    rows, n, r = 6000, 256, 64
    x, dy = rows16(rnd(1, rows, n), T[kind]), rows16(rnd(2, rows, n), T[kind])
    s, u = rnd(3, rows, r).float().cuda(), rnd(4, rows, r).float().cuda()
    at, none = ints([0, 1000, rows]), ints([-1, -1])
    w = rows16(rnd(5, 2, n, n) / 16, T[kind])
    da, db = rnd(6, 3, r, n).float().cuda(), rnd(7, 3, n, r).float().cuda()
    a0, b0 = da.clone(), db.clone()
    want = mma.gemm_grouped(x, w, at)
    for _ in range(20):
        mma.gemm_lora_wgrad(dy, x, s, u, at, none, adapters_total=3, dA=da, dB=db, accumulate=True)
        # (results in the memory that the call above has given back)
        got = [mma.gemm_grouped(x, w, at) for _ in range(3)]
        assert all(torch.equal(g, want) for g in got)
        del got
    assert torch.equal(da, a0) and torch.equal(db, b0)
    # no rows at all
    mma.gemm_lora_wgrad(dy[:0], x[:0], s[:0], u[:0], ints([0, 0, 0]), none, adapters_total=3, dA=da, dB=db, accumulate=True)
    assert torch.equal(da, a0) and torch.equal(db, b0)
    za, zb = mma.gemm_lora_wgrad(dy, x, s, u, at, none, adapters_total=3)
    assert not za.any() and not zb.any()
