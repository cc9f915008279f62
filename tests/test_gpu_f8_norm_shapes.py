"""The norm, its gradient and the quantiser at sizes where every block works
through several rows or tiles in turn, in each of the register and ring shapes,
against the definitions in 64 bits.

Tolerances as beside the small sizes: FP32 sums of a row are within 2^-17 of
exact, y within 2^-17, scales 2^-16; an 8-bit value is within half a step of
the exact quotient by its scale (2^-4 relative for E4M3, 2^-3 for E5M2, or half
the smallest step), with those errors on top.  The weight's gradient adds up
the rows in FP32: some 20 per block, 456 blocks by twos and a tree, below 2^-18
of the sum of magnitudes, and 2^-17 from 1 / rms.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half an ulp
CODE = {"f16": 1, "bf16": 2, "f32": 5}
F8 = {"e4m3": (448.0, 2.0 ** -4, 2.0 ** -10), "e5m2": (57344.0, 2.0 ** -3, 2.0 ** -17)}
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def rows16(seed, m, n, dtype, scale=1.0):
    """Random rows on 16-byte boundaries, NaN in the gaps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = 16 // dtype.itemsize
    big = torch.full((m, -(-n // per) * per + per), float("nan"), dtype=dtype, device="cuda")
    big[:, :n] = (scale * torch.randn(m, n, generator=g, device="cuda")).to(dtype)
    return big[:, :n]


def blocks64(y, rows):
    """Largest magnitude of each block of rows x 128."""
    m, n = y.shape
    big = y.new_zeros(-(-m // rows) * rows, -(-n // 128) * 128)
    big[:m, :n] = y.abs()
    return big.view(-(-m // rows), rows, -(-n // 128), 128).amax((1, 3))


def check_f8(q, s, y, fmt, rows, rel):
    top, half, low = F8[fmt]
    m, n = y.shape
    want = (blocks64(y, rows) / top).clamp_min(TINY)
    assert s.shape == want.shape
    assert bool(((s.double() - want).abs() <= want * rel).all())
    v = y / s.double().repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :n]
    bound = torch.clamp_min(v.abs() * half, low) * (1 + 2.0 ** -8) + v.abs() * rel
    assert bool(((q.double() - v).abs() <= bound).all())


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", [(2000, 1500), (2000, 3000), (1999, 5000), (2000, 5555), (2000, 8192),
                                 (1000, 12001), (1000, 16384), (701, 128)])
@pytest.mark.parametrize("res", [False, True])
def test_norm(t, m, n, res):
    dt = T[t]
    x = rows16(1, m, n, dt)
    r = rows16(2, m, n, dt, 2.0) if res else None
    w = (1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(3))).to(dt).cuda()
    q, s, h, y = mma.rmsnorm_f8(x, w, r, eps=1e-5, y=True)
    h64 = x.double() + (r.double() if res else 0.0)
    y64 = h64 * w.double() / torch.sqrt((h64 ** 2).mean(1, keepdim=True) + 1e-5)
    assert bool(((h.double() - h64).abs() <= h64.abs() * (U[t] + 2.0 ** -23) + 2.0 ** -25).all())
    assert bool(((y.double() - y64).abs() <= y64.abs() * (U[t] + 2.0 ** -17) + 2.0 ** -25).all())
    check_f8(q, s, y64, "e4m3", 1, 2.0 ** -16)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", [(2000, 2500), (2000, 4096), (1300, 5000), (1000, 7168), (2000, 8192),
                                 (1000, 12001), (700, 16384)])
@pytest.mark.parametrize("res", [False, True])
def test_norm_backward(t, m, n, res):
    dt = T[t]
    dy, h = rows16(11, m, n, dt), rows16(12, m, n, dt)
    dh = rows16(13, m, n, dt) if res else None
    w = (1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(14))).to(dt).cuda()
    dx, dw = mma.rmsnorm_backward(dy, h, w, dh, eps=1e-5)
    d, k, v = dy.double(), h.double(), w.double()
    rms = torch.sqrt((k ** 2).mean(1, keepdim=True) + 1e-5)
    g = d * v
    want = g / rms - k * (g * k).mean(1, keepdim=True) / rms ** 3
    mag = g.abs() / rms + k.abs() * (g * k).abs().mean(1, keepdim=True) / rms ** 3
    if res:
        want = want + dh.double()
        mag = mag + dh.double().abs()
    assert bool(((dx.double() - want).abs() <= mag * 2.0 ** -16 + want.abs() * U[t] + 2.0 ** -25).all())
    want_w, mag_w = (d * k / rms).sum(0), (d * k / rms).abs().sum(0)
    assert bool(((dw.double() - want_w).abs() <= mag_w * 2.0 ** -16).all())
    # the same bits in place, over dy and over the residual path's gradient
    need = binding.load().mma_rmsnorm_backward_workspace(m, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for which in ("dy", "dh")[:1 + res]:
        a = {"dy": rows16(11, m, n, dt), "dh": rows16(13, m, n, dt) if res else None}
        dw2 = torch.empty(n, device="cuda")
        rc = binding.load().mma_rmsnorm_backward(
            CODE[t], CODE[t], m, n, a["dy"].data_ptr(), a["dy"].stride(0), h.data_ptr(), h.stride(0),
            w.data_ptr(), 1e-5, a["dh"].data_ptr() if res else None, a["dh"].stride(0) if res else 0,
            a[which].data_ptr(), a[which].stride(0), dw2.data_ptr(), ws.data_ptr(), need,
            torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0
        assert bool((a[which] == dx).all()) and bool((dw2 == dw).all())


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
@pytest.mark.parametrize("m,n", [(4000, 2051), (2051, 4000), (9000, 2048)])
def test_quantise(t, fmt, rows, transpose, m, n):
    x = rows16(31, m, n, T[t], 3.0)
    q, s = mma.quantize_f8(x, fmt=fmt, block_rows=rows, transpose=transpose)
    x64 = x.double().t() if transpose else x.double()
    check_f8(q, s, x64, fmt, rows, 2.0 ** -24)
