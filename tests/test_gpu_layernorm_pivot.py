"""The layer norm's sums about a pivot where that is far from the mean: the row's samples
are numbers of 2^66 among zeros, so that the squares are beyond FP32.  In FP32, mean first,
the variance is infinite and 1 / std zero: y is the bias, and dx and the row's share of dw
are zeros, however many rows there are.  Another row stands among them, with the
tolerances of the other tests of the layer norm: z within 2^-16 (1 + far) (1 + |z|), far =
mean |h| / std < 1; a gradient's terms within 2^-15 (1 + far) of their magnitudes.
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


def rows(m, n, kind):
    """Rows whose numbers of 2^66 stand where the row is sampled."""
    x = torch.zeros(m, n, dtype=torch.float64)
    q, lane = n // 32, torch.arange(32)
    x[:, lane * q + 2 * lane % q] = 2.0 ** 66
    x[1::2] = -x[1::2]
    x[2] = torch.randn(n, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    return x.to(kind).cuda()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(5, 4096), (400, 4096), (400, 1000), (1300, 264), (5, 20000), (200, 17000)])
def test_forward(m, n, kind):
    x = rows(m, n, kind)
    w = torch.ones(n, dtype=kind, device="cuda")
    b = torch.randn(n, generator=torch.Generator().manual_seed(3)).to(kind).cuda()
    y, _ = mma.layernorm(x, w, b)
    far = torch.arange(m, device="cuda") != 2
    assert torch.equal(y[far], b.expand(m, n)[far])
    h = x[2].double()
    z = (h - h.mean()) / ((h - h.mean()).square().mean() + 1e-5).sqrt()
    u = torch.finfo(kind).eps / 2
    want = z + b.double()
    assert bool(((y[2].double() - want).abs() <= want.abs() * u + 2.0 ** -15 * (1 + z.abs())).all())


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(5, 4096), (400, 1000), (1300, 264), (5, 20000)])
def test_gradient(m, n, kind):
    x = rows(m, n, kind)
    dy = torch.randn(m, n, generator=torch.Generator().manual_seed(2)).to(kind).cuda()
    w = torch.ones(n, dtype=kind, device="cuda")
    dx, dw, db = mma.layernorm_backward(dy, x, w)
    far = torch.arange(m, device="cuda") != 2
    assert not dx[far].any()
    h, g = x[2].double(), dy[2].double()
    c = h - h.mean()
    std = (c.square().mean() + 1e-5).sqrt()
    z, gm = c / std, g - g.mean()
    want = (gm - z * (gm * z).mean()) / std
    mag = (g.abs() + g.abs().mean() + z.abs() * (g.abs() * z.abs()).mean()) / std
    u = torch.finfo(kind).eps / 2
    assert bool(((dx[2].double() - want).abs() <= want.abs() * u + 2.0 ** -14 * mag).all())
    assert bool(((dw.double() - g * z).abs() <= 2.0 ** -14 * g.abs() * (1 + z.abs())).all())
    every = dy.double()
    assert bool(((db.double() - every.sum(0)).abs() <= 2.0 ** -16 * every.abs().sum(0)).all())
