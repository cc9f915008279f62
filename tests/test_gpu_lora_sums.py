"""The rows' sums of products with adapters where they run over many k's."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding
from test_gpu_lora import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("rows", [4000, 16384])
def test_sums_of_long_rows(rows, row):
    """Terms of one sign.  The tensor cores drop low bits of a sum in each step, up to
    2^-22 of it: over 64 k's, four steps, 2^-20.  Up to 256 of these are added to
    nearest, 2^-24 of a sum that grows: 256 / 2 of those, 2^-17."""
    k, r = 16384, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.rand(rows, k, generator=g, device="cuda").bfloat16()
    a = torch.rand(2, r, k, generator=g, device="cuda").bfloat16()
    w = torch.zeros(64, k, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(2, 64, r, dtype=torch.bfloat16, device="cuda")
    at = [0, rows - 1000, rows]
    if row:
        _, s = mma.gemm_lora(x, w.t().contiguous(), a.transpose(1, 2).contiguous(), b.transpose(1, 2).contiguous(),
                             ints(at), b_layout="row", sums=True)
    else:
        _, s = mma.gemm_lora(x, w, a, b, ints(at), sums=True)
    for j in range(2):
        for i in range(at[j], at[j + 1], 4096):
            i1 = min(i + 4096, at[j + 1])
            want = x[i:i1].double() @ a[j].double().t()
            assert bool(((s[i:i1].double() - want).abs() <= want * (2.0 ** -17 + 2.0 ** -20)).all())
