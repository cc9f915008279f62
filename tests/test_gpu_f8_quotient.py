"""8-bit values are the FP32 quotient x / s rounded to nearest, ties to even,
bit for bit: the quotient often lies half-way between two 8-bit values, where
a product with the reciprocal of s goes the wrong way.  No tolerance.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed),
                       device="cuda")


def bits(x, s, rows, fmt):
    """The bits of x over its block's scale, in plain torch."""
    f8, most = F8[fmt]
    m, n = x.shape
    s = s.repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :n]
    return (x.float() / s).clamp(-most, most).to(f8).view(torch.uint8)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantiser(t, fmt, rows, transpose):
    x = (rnd(1, 1000, 1416) * torch.exp(2 * rnd(2, 1000, 1))).to(T[t])
    for cut in (x, x[:257, :1304]):
        q, s = mma.quantize_f8(cut, fmt=fmt, block_rows=rows, transpose=transpose)
        want = bits(cut.t() if transpose else cut, s, rows, fmt)
        assert bool((q.view(torch.uint8) == want).all())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantiser_over_the_range_of_scales(fmt, rows, transpose):
    """Blocks from FP32's smallest numbers to its largest, zeros of both signs
    among them."""
    x = rnd(3, 1024, 1024)
    e = torch.linspace(-148, 125, 64, device="cuda").round().view(8, 8)
    x = (x / x.abs().max()).double() * torch.exp2(e.double()).repeat_interleave(128, 0).repeat_interleave(128, 1)
    x = x.float()
    x[5::17, 3::11] = 0.0
    x[7::19, 4::13] = -0.0
    q, s = mma.quantize_f8(x, fmt=fmt, block_rows=rows, transpose=transpose)
    assert bool((q.view(torch.uint8) == bits(x.t() if transpose else x, s, rows, fmt)).all())


@pytest.mark.parametrize("m,n", [(3, 4096), (700, 1000), (520, 3000), (300, 8192), (2, 16400)])
def test_norm(m, n):
    """y in FP32 is what the 8-bit values are made of."""
    x, r = rnd(4, m, n), rnd(5, m, n)
    w = 1 + 0.1 * rnd(6, n)
    q, s, _, y = mma.rmsnorm_f8(x, w, r, y=True)
    assert bool((q.view(torch.uint8) == bits(y, s, 1, "e4m3")).all())


def test_ties():
    """Values 7.25 i / 256 for odd i: over s, which is 7.25 / 448 rounded, they
    are 1.75 i, many of them half-way between two E4M3 values."""
    x = torch.zeros(1, 128, device="cuda")
    x[0, 0] = 7.25
    x[0, 1:127] = 7.25 * (torch.arange(1, 127, device="cuda") * 2 + 1) / 256
    q, s = mma.quantize_f8(x)
    assert bool((q.view(torch.uint8) == bits(x, s, 1, "e4m3")).all())
