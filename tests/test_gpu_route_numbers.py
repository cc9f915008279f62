"""The router's gradient where logits are NaN or infinite."""
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


@pytest.mark.parametrize("t,e", [(40, 70), (40, 5), (1000, 256), (300, 1000)])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_of_bad_logits(t, e, normalize):
    """A token whose logits hold a NaN or +inf has weights of NaN, and so its gradient;
    the others' are as without it, but for the counts of its choices."""
    g = torch.Generator().manual_seed(t)
    x = torch.randn(t, e, generator=g).cuda()
    x[3] = float("nan")
    x[5] = -float("inf")
    x[5, 2] = float("nan")
    x[7, 4] = float("nan")
    x[9, 1] = float("inf")
    x[11] = float("nan")  # masked
    x[13] = -float("inf")  # without any expert
    mask = torch.ones(t, dtype=torch.bool, device="cuda")
    mask[11] = False
    r = mma.route(x, 3, mask=mask, normalize=normalize)
    dw = torch.randn(t, 3, generator=g).cuda()
    dx = mma.route_backward(x, r, dw, mask=mask, normalize=normalize)
    bad = [3, 5, 7, 9]
    assert bool(r.weights[bad][r.experts[bad] >= 0].isnan().all())
    for i in bad:
        assert bool(dx[i].isnan().all()), i
    assert not dx[11].any() and not dx[13].any()
    keep = torch.ones(t, dtype=torch.bool)
    keep[bad] = False
    clean = torch.where(keep.cuda()[:, None], x, torch.zeros_like(x))
    again = mma.route_backward(clean, mma.route(clean, 3, mask=mask, normalize=normalize), dw, mask=mask, normalize=normalize)
    assert torch.equal(dx[keep.cuda()], again[keep.cuda()])
