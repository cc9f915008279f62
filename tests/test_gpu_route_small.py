"""The router's probabilities far below the largest."""
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


@pytest.mark.parametrize("shifted", [False, True])
@pytest.mark.parametrize("tokens", [50, 3000])
def test_small_probabilities(tokens, shifted):
    """Distances of up to 85 to the largest logit.  The special function is off by two
    units in the last place at most, 2^-22, as is the division; the argument by 2^-23,
    and the sum of four by three roundings, 2^-22, and its terms' 2^-21: below 2^-19.
    Where the largest logit is not zero the distance d itself is rounded, by 2^-24 of it,
    and e^d is off by 2^-24 d (1 + 2^-16) more, as the largest of the sum's terms is not."""
    g = torch.Generator().manual_seed(tokens)
    x = -85 * torch.rand(tokens, 4, generator=g)
    x[:, 1] = 0
    x = x.cuda() + shifted * torch.randn(tokens, 1, generator=g).cuda()
    got = mma.route(x, 4, normalize=False)
    at = got.experts.long()
    p = torch.softmax(x.double(), 1).gather(1, at)
    d = (x.double().amax(1, keepdim=True) - x.double()).gather(1, at)
    # (a small term's rounding reaches the sum with its share of it)
    rel = 2.0 ** -19 + shifted * 2.0 ** -23.9 * (d + (p * d).sum(1, keepdim=True))
    assert bool(((got.weights.double() - p).abs() <= p * rel).all())
    # and in the gradient, of the third choice's weight: p_e (1_e3 - p_3)
    dw = torch.zeros(tokens, 4, device="cuda")
    dw[:, 2] = 1
    dx = mma.route_backward(x, got, dw, normalize=False).double().gather(1, at)
    want = p * (dw.double() - p[:, 2:3])
    lim = want.abs() * (2.0 ** -19 + rel + rel[:, 2:3])
    assert bool(((dx - want).abs() <= lim + 2.0 ** -126).all())
