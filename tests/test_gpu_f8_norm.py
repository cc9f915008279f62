"""The norm with an 8-bit output, its gradient and the quantiser, against the
definitions in 64 bits.

Tolerances.  FP32 sums of a row run over at most 64 terms per thread and ten
levels of a tree, so they are within 2^-17 of exact for sums of squares; y
has half of that plus five roundings, below 2^-17.  A scale is y's largest
magnitude over 448 and inherits 2^-17 + 2^-23.  An 8-bit value is within
half a step of y / s (2^-4 relative for E4M3, 2^-3 for E5M2, and half the
smallest step below the normal numbers), with those errors on top.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half an ulp
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10),
      "e5m2": (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def rnd(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def rows16(x, dtype, pad=0):
    """x on the GPU with rows on 16-byte boundaries, `pad` more 16-byte
    chunks between them, and NaN in the gaps."""
    m, n = x.shape
    per = 16 // torch.empty((), dtype=dtype).element_size()
    big = torch.full((m, -(-n // per) * per + pad * per), float("nan"), dtype=dtype,
                     device="cuda")
    big[:, :n] = x.to(dtype)
    return big[:, :n]


def scales64(y, rows, fmax, pow2):
    m, n = y.shape
    out = torch.zeros(-(-m // rows), -(-n // 128), dtype=torch.float64)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = y[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128].abs().max() / fmax
    out = out.clamp_min(TINY)
    return torch.exp2(torch.ceil(torch.log2(out))) if pow2 else out


def spread(s, rows, m, n):
    return s.repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :n]


def check_f8(q, s, y, fmt, rows, rel, what):
    """q, s stand for y (64 bits), whose FP32 form may be off by `rel`."""
    _, fmax, half, sub = F8[fmt]
    m, n = y.shape
    sf = spread(s.double().cpu(), rows, m, n)
    v = y / sf
    err = (q.double().cpu() - v).abs()
    bound = torch.maximum(v.abs() * half, torch.tensor(sub, dtype=torch.float64)) * (1 + 2.0 ** -8) \
        + v.abs() * rel
    assert bool((err <= bound).all()), f"{what}: {float((err / bound).max())}"


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 128), (3, 4096), (5, 1000), (7, 33), (2, 8),
                                 (4, 5000), (130, 256), (2, 7168), (3, 16400), (2, 40001)])
def test_norm(t, m, n):
    dt = T[t]
    x, r = rows16(rnd(1, m, n), dt, 1), rows16(2 * rnd(2, m, n), dt)
    for w32, res, pow2 in ((False, True, False), (True, False, True)):
        w = (1 + 0.1 * rnd(3, n)).to(torch.float32 if w32 else dt).cuda()
        q, s, h, y = mma.rmsnorm_f8(x, w, r if res else None, eps=1e-5, pow2=pow2, y=True)
        h64 = x.double().cpu() + (r.double().cpu() if res else 0.0)
        y64 = h64 * w.double().cpu() / torch.sqrt((h64 ** 2).mean(1, keepdim=True) + 1e-5)
        if res:
            hr = h.double().cpu()
            assert bool(((hr - h64).abs() <= h64.abs() * (U[t] + 2.0 ** -23) + 2.0 ** -25).all())
        else:
            assert h is x
        err = (y.double().cpu() - y64).abs()
        assert bool((err <= y64.abs() * (U[t] + 2.0 ** -17) + 2.0 ** -25).all())
        if pow2:
            mant, _ = torch.frexp(s.cpu())
            assert bool((mant == 0.5).all())
            s64 = scales64(y64, 1, 448.0, False)
            ratio = s.double().cpu() / s64
            assert bool(((ratio >= 1 - 2.0 ** -16) & (ratio <= 2 * (1 + 2.0 ** -16))).all())
        else:
            s64 = scales64(y64, 1, 448.0, False)
            assert bool(((s.double().cpu() - s64).abs() <= s64 * 2.0 ** -16).all())
        check_f8(q, s, y64, "e4m3", 1, 2.0 ** -16, f"{t} {m}x{n}")
        assert s.shape == (m, -(-n // 128))


def test_norm_special_rows():
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(5)).cuda().to(torch.bfloat16)
    x = rows16(x.double().cpu(), torch.bfloat16)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 299] = float("inf")
    w = torch.ones(300, dtype=torch.bfloat16, device="cuda")
    w[140] = float("inf")
    q, s, h = mma.rmsnorm_f8(x, w, rows16(torch.zeros(6, 300), torch.bfloat16), eps=1e-6)
    q, s = q.float().cpu(), s.cpu()
    # zeros: 0 * inf is NaN in block 1, the other blocks are exact zeros
    assert bool((q[1, :128] == 0).all()) and float(s[1, 0]) == TINY
    assert bool(torch.isnan(s[1, 1])) and bool((q[1, 256:] == 0).all())
    # a NaN or infinite element: rms is NaN or infinite, for the whole row
    assert bool(torch.isnan(q[2]).all()) and bool(torch.isnan(s[2]).all())
    assert bool(torch.isnan(q[3, 299])) and bool(torch.isnan(s[3, 2]))
    # an infinite weight: its block has an infinite scale
    assert bool(torch.isinf(s[0, 1])) and bool((q[0, 128:140] == 0).all())
    assert bool(torch.isfinite(s[0, 0])) and bool(torch.isfinite(q[0, :128]).all())
    # large values stay finite in FP32
    big = rows16(torch.full((1, 256), 3e38, dtype=torch.float64), torch.float32)
    _, s2, _, y2 = mma.rmsnorm_f8(big, torch.ones(256, device="cuda"), eps=0.0, y=True)
    assert bool((y2.cpu() == 0).all())  # mean of squares overflows: 1 / rms is 0


def test_norm_in_place_and_guards():
    m, n, ldb = 5, 200, 208
    x, r = rows16(rnd(8, m, n), torch.bfloat16), rows16(rnd(9, m, n), torch.bfloat16)
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    q0, s0, h0 = mma.rmsnorm_f8(x, w, r)
    # the sum into the residual itself; Q in a buffer of canaries
    buf = torch.full((m + 2, 256), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.full((m + 2, 2), -7.0, device="cuda")
    r2 = r.clone(memory_format=torch.preserve_format)
    r2 = rows16(r.double().cpu(), torch.bfloat16)
    rc = binding.load().mma_rmsnorm_f8(
        2, 2, m, n, x.data_ptr(), x.stride(0), r2.data_ptr(), r2.stride(0), w.data_ptr(), 1e-6, 0,
        r2.data_ptr(), r2.stride(0), None, 0, buf[1:].data_ptr(), 256, st[1:].data_ptr(), 2, 1, None)
    torch.cuda.synchronize()
    assert rc == 0
    assert bool((r2 == h0).all()) and bool((st[1:-1] == s0).all())
    assert bool((buf[1:-1, :n] == q0.view(torch.uint8)).all())
    assert bool((buf[0] == 0xA5).all()) and bool((buf[-1] == 0xA5).all())
    assert bool((buf[1:-1, n:] == 0xA5).all()) and bool((st[0] == -7).all())
    assert bool((st[-1] == -7).all())


def backward64(dy, h, w, dh, eps):
    n = h.shape[1]
    rms = torch.sqrt((h ** 2).mean(1, keepdim=True) + eps)
    g = dy * w
    dx = g / rms - h * (g * h).sum(1, keepdim=True) / (n * rms ** 3)
    return dx + (0 if dh is None else dh), (dy * h / rms).sum(0)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (700, 33), (3, 4096), (1000, 1000), (5, 16400), (4, 40001)])
@pytest.mark.parametrize("res", [False, True])
def test_norm_backward(t, m, n, res):
    dt = T[t]
    dy, h = rows16(rnd(11, m, n), dt), rows16(rnd(12, m, n), dt, 1)
    dh = rows16(rnd(13, m, n), dt) if res else None
    w = (1 + 0.1 * rnd(14, n)).to(dt).cuda()
    dx, dw = mma.rmsnorm_backward(dy, h, w, dh, eps=1e-5)
    d64 = [a.double().cpu() for a in (dy, h, w)]
    want, want_w = backward64(*d64, None if dh is None else dh.double().cpu(), 1e-5)
    # terms of dx: g / rms, its projection (whose sum may cancel: bounded by
    # the sum of magnitudes) and the residual's gradient
    rms = torch.sqrt((d64[1] ** 2).mean(1, keepdim=True) + 1e-5)
    g = (d64[0] * d64[2]).abs() / rms
    proj = d64[1].abs() * ((d64[0] * d64[2] * d64[1]).abs().mean(1, keepdim=True)) / rms ** 3
    mag = g + proj + (0 if dh is None else dh.double().cpu().abs())
    err = (dx.double().cpu() - want).abs()
    assert bool((err <= mag * 2.0 ** -16 + want.abs() * U[t] + 2.0 ** -25).all())
    magw = (d64[0] * d64[1] / rms).abs().sum(0)
    assert bool(((dw.double().cpu() - want_w).abs() <= magw * 2.0 ** -16).all())
    again = mma.rmsnorm_backward(dy, h, w, dh, eps=1e-5)
    assert bool((again[0] == dx).all()) and bool((again[1] == dw).all())


def test_norm_backward_against_differences():
    """dX and dW against central differences of the forward's formula: for
    L = sum(dy * y) in 64 bits, step 1e-4, the differences' own error is of
    the order of 1e-8."""
    m, n, eps = 2, 37, 1e-3
    dy, h, w = rnd(21, m, n), rnd(22, m, n), 1 + 0.1 * rnd(23, n)
    dy, h, w = (a.float().double() for a in (dy, h, w))

    def loss(h, w):
        return float((dy * h * w / torch.sqrt((h ** 2).mean(1, keepdim=True) + eps)).sum())

    dx, dw = mma.rmsnorm_backward(rows16(dy, torch.float32), rows16(h, torch.float32),
                                  w.float().cuda(), eps=eps)
    for i, j in ((0, 0), (1, 36), (0, 17)):
        d = torch.zeros_like(h)
        d[i, j] = 1e-4
        assert abs((loss(h + d, w) - loss(h - d, w)) / 2e-4 - float(dx[i, j])) < 1e-4
    for j in (0, 20, 36):
        d = torch.zeros_like(w)
        d[j] = 1e-4
        assert abs((loss(h, w + d) - loss(h, w - d)) / 2e-4 - float(dw[j])) < 1e-4


@pytest.mark.parametrize("n", [200, 1000, 16400])
def test_norm_backward_in_place(n):
    """dX over dY, and over the residual path's gradient, rows of one stride."""
    m = 700
    dy, h, r = (rows16(rnd(50 + i, m, n), torch.bfloat16) for i in range(3))
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    want, want_w = mma.rmsnorm_backward(dy, h, w, r)
    need = binding.load().mma_rmsnorm_backward_workspace(m, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for which in ("dy", "r"):
        a = {"dy": rows16(dy.double().cpu(), torch.bfloat16),
             "r": rows16(r.double().cpu(), torch.bfloat16)}
        dw = torch.empty(n, device="cuda")
        rc = binding.load().mma_rmsnorm_backward(
            2, 2, m, n, a["dy"].data_ptr(), a["dy"].stride(0), h.data_ptr(), h.stride(0),
            w.data_ptr(), 1e-6, a["r"].data_ptr(), a["r"].stride(0), a[which].data_ptr(),
            a[which].stride(0), dw.data_ptr(), ws.data_ptr(), need, None)
        torch.cuda.synchronize()
        assert rc == 0
        assert bool((a[which] == want).all()) and bool((dw == want_w).all())


def test_norm_backward_without_rows():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    dx, dw = mma.rmsnorm_backward(z, z, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 300), (128, 128), (130, 257), (1000, 24), (17, 2000)])
def test_quantize(t, fmt, rows, transpose, m, n):
    x = rows16(rnd(31, m, n) * torch.exp(2 * rnd(32, 1, n)), T[t], 1)
    x64 = x.double().cpu()
    x64 = x64.t() if transpose else x64
    for pow2 in (False, True):
        q, s = mma.quantize_f8(x, fmt=fmt, block_rows=rows, transpose=transpose, pow2=pow2)
        assert q.dtype == F8[fmt][0] and tuple(q.shape) == tuple(x64.shape)
        # the largest magnitude is exact, so the scale is one division off
        s64 = scales64(x64, rows, F8[fmt][1], pow2)
        assert tuple(s.shape) == tuple(s64.shape)
        assert bool(((s.double().cpu() - s64).abs() <= s64 * (0 if pow2 else 2.0 ** -24)).all())
        check_f8(q, s, x64, fmt, rows, 2.0 ** -22, f"{t} {fmt} {rows} {transpose} {m}x{n}")
        if pow2:  # x / s is exact: the value is the one nearest to it
            v = (x64 / spread(s64, rows, *x64.shape)).float()
            assert bool((q.float().cpu() == v.to(F8[fmt][0]).float()).all())


def test_quantize_special_blocks():
    x = torch.zeros(4, 512, device="cuda")
    x[0, 5] = float("nan")
    x[0, 130] = float("inf")
    x[1, 0] = 1e-44          # its quotient by 448 underflows
    x[2, 0:128] = 3.0e38
    for rows in (1, 128):
        q, s = mma.quantize_f8(x, block_rows=rows)
        q, s = q.float().cpu(), s.cpu()
        assert bool(torch.isnan(s[0, 0])) and bool(torch.isinf(s[0, 1]))
        assert bool(torch.isnan(q[0, :128]).all()) and bool(torch.isnan(q[0, 130]))
        assert float(s[0, 2]) == TINY and bool((q[0, 256:] == 0).all())
        if rows == 1:
            assert float(s[1, 0]) == TINY and bool((q[1] == 0).all())
            assert bool((q[2, :128] == 448).all())
            assert bool((q[0, 131:256] == 0).all())


def test_quantize_guards():
    """Nothing outside the result is written, at sizes that end inside every
    tile, and scales of any strides are placed by them."""
    for transpose, rows in ((False, 1), (False, 128), (True, 1), (True, 128)):
        m, n = 131, 141
        x = rows16(rnd(41, m, n), torch.bfloat16)
        q0, s0 = mma.quantize_f8(x, block_rows=rows, transpose=transpose)
        a, b = (n, m) if transpose else (m, n)
        buf = torch.full((a + 2, 160), 0xA5, dtype=torch.uint8, device="cuda")
        st = torch.full((s0.shape[0] + 2, 3), -7.0, device="cuda")
        rc = binding.load().mma_quantize_f8(2, 7, m, n, rows, int(transpose), 0, x.data_ptr(),
                                            x.stride(0), buf[1:].data_ptr(), 160,
                                            st[1:].data_ptr(), 3, 1, None)
        torch.cuda.synchronize()
        assert rc == 0
        assert bool((buf[1:-1, :b] == q0.view(torch.uint8)).all())
        assert bool((buf[0] == 0xA5).all()) and bool((buf[-1] == 0xA5).all())
        assert bool((buf[1:-1, b:] == 0xA5).all())
        assert bool((st[1:-1, :2] == s0).all()) and bool((st[:, 2] == -7).all())
        assert bool((st[0] == -7).all()) and bool((st[-1] == -7).all())
