"""The example layer's router on the GPU against the definition, and its reference, which
does without it."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from mixed_precision_dense_02_gb300 import expert_layer
from test_expert_layer_route import check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import binding, build
    build.build()
    yield
    binding.device_status()


@pytest.mark.parametrize("t,e,k", [(1, 4, 1), (300, 8, 2), (7, 50, 40), (3, 1500, 5), (40, 1024, 32)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_route(t, e, k, kind):
    x = logits(t, e, kind).cuda()
    check(expert_layer.route(x, k), x.cpu(), k)
    check(expert_layer.plain_route(x, k), x.cpu(), k)
    check(expert_layer.route(x.t().contiguous().t(), k), x.cpu(), k)


def test_gradient_through_the_weights():
    x = logits(9, 6, torch.float32).cuda().requires_grad_()
    expert_layer.route(x, 2)[2].square().sum().backward()
    assert float(x.grad.abs().sum()) > 0


def test_reference_does_without_the_router(monkeypatch):
    w = expert_layer.Weights(8, 128, 64)
    x, r = (torch.randn(50, 128, generator=torch.Generator().manual_seed(i)).cuda().bfloat16() for i in (1, 2))
    want = expert_layer.reference(x, r, w)

    def refuse(*a, **k):
        raise AssertionError("the reference calls the router under test")

    monkeypatch.setattr(expert_layer.mma, "route", refuse)
    assert torch.equal(expert_layer.reference(x, r, w), want)
