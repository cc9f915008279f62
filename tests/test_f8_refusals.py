"""Refusals of the 8-bit and grouped calls, without a GPU: what the C ABI and
the Python binding reject before a device is touched."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding, build

F16, BF16, I8, F64, F32, I32, E4M3, E5M2 = range(1, 9)
OK, INVALID, UNSUP, MISAL, LAUNCH, TIMEOUT, NODEV = range(7)
P, Q, R = 1 << 20, 1 << 24, 1 << 26  # fake aligned addresses; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def nodev():
    return OK if torch.cuda.is_available() else NODEV


def call(fn, args, kw):
    for k, v in kw.items():
        assert k in args, k
        args[k] = v
    return getattr(binding.load(), fn)(*args.values(), None)


def norm(**kw):
    return call("mma_rmsnorm_f8", dict(
        type=BF16, wt=BF16, M=4, N=256, X=P, ldx=256, R=P, ldr=256, W=P, eps=1e-6, pow2=0, H=Q,
        ldh=256, Y=0, ldy=0, Q=R, ldq=256, S=R, srow=1, sblk=4), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=I8), UNSUP), (dict(wt=F16), UNSUP), (dict(type=F32), UNSUP),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(X=0), INVALID), (dict(W=0), INVALID),
    (dict(ldx=255), INVALID), (dict(ldr=8), INVALID), (dict(ldh=8), INVALID),
    (dict(ldq=128), INVALID), (dict(S=0), INVALID), (dict(srow=-1), INVALID),
    (dict(Q=0, Y=0), INVALID), (dict(H=P, ldh=512), INVALID),
    (dict(X=P + 8), MISAL), (dict(ldx=257), MISAL), (dict(W=P + 2), MISAL),
    (dict(Q=R + 4), MISAL), (dict(ldq=264), MISAL), (dict(S=R + 2), MISAL),
    (dict(Y=Q, ldy=260), MISAL), (dict(M=0, X=0, Q=0, W=0), OK), (dict(N=0, X=0), OK),
])
def test_norm(kw, code):
    assert norm(**kw) == code


def back(**kw):
    return call("mma_rmsnorm_backward", dict(
        type=BF16, wt=F32, M=4, N=256, DY=P, lddy=256, H=P, ldh=256, W=P, eps=1e-6, R=0, ldr=0,
        DX=Q, lddx=256, DW=R, ws=R, bytes=1 << 20), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=E4M3), UNSUP), (dict(wt=F16), UNSUP), (dict(M=-2), INVALID),
    (dict(DY=0), INVALID), (dict(H=0), INVALID), (dict(DX=0), INVALID), (dict(DW=0), INVALID),
    (dict(lddx=128), INVALID), (dict(ws=0), INVALID), (dict(bytes=4 * 256 * 4 - 1), INVALID),
    (dict(DX=P, lddx=512), INVALID), (dict(R=Q, ldr=8), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(DW=R + 2), MISAL), (dict(H=P + 4), MISAL), (dict(ldh=260), MISAL), (dict(N=0), OK),
])
def test_norm_backward(kw, code):
    assert back(**kw) == code


def test_norm_backward_workspace():
    f = binding.load().mma_rmsnorm_backward_workspace
    assert f(0, 4096) == 0 and f(4, 256) == 4 * 256 * 4
    assert f(10 ** 6, 256) == 456 * 256 * 4 and f(-1, 5) == 0


def quant(**kw):
    return call("mma_quantize_f8", dict(
        type=F32, f8=E4M3, M=130, N=260, rows=1, trans=0, pow2=0, X=P, ldx=260, Q=Q, ldq=272, S=R,
        srow=1, sblk=130), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=F64), UNSUP), (dict(f8=BF16), UNSUP), (dict(rows=64), INVALID),
    (dict(rows=0), INVALID), (dict(M=-1), INVALID), (dict(X=0), INVALID), (dict(Q=0), INVALID),
    (dict(ldx=200), INVALID), (dict(ldq=256), INVALID), (dict(trans=1, ldq=128), INVALID),
    (dict(S=0), INVALID), (dict(sblk=-1), INVALID), (dict(ldx=261), MISAL),
    (dict(ldq=264), MISAL), (dict(Q=Q + 1), MISAL), (dict(S=R + 1), MISAL),
    (dict(M=0, X=0, Q=0, S=0), OK),
])
def test_quantize(kw, code):
    assert quant(**kw) == code


def f8(**kw):
    return call("mma_gemm_f8", dict(
        ta=E4M3, tb=E5M2, td=BF16, M=64, N=130, K=256, A=P, lda=256, SA=R, sarow=1, sablk=64,
        B=P, ldb=256, SB=R, rows=128, sbrow=1, sbblk=2, C=0, ldc=0, D=Q, ldd=130), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(ta=I8), UNSUP), (dict(tb=BF16), UNSUP), (dict(td=I32), UNSUP), (dict(td=E4M3), UNSUP),
    (dict(rows=2), INVALID), (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(A=0), INVALID),
    (dict(B=0), INVALID), (dict(D=0), INVALID), (dict(SA=0), INVALID), (dict(SB=0), INVALID),
    (dict(lda=255), INVALID), (dict(ldb=128), INVALID), (dict(ldd=129), INVALID),
    (dict(C=P, ldc=100), INVALID), (dict(C=Q, ldc=136), INVALID), (dict(sarow=-1), INVALID),
    (dict(sbblk=-2), INVALID), (dict(A=P + 8), MISAL), (dict(lda=264), MISAL),
    (dict(ldb=260), MISAL), (dict(SA=R + 2), MISAL), (dict(D=Q + 1), MISAL),
    (dict(M=0, A=0, D=0), OK), (dict(N=0, B=0, D=0), OK),
])
def test_f8(kw, code):
    assert f8(**kw) == code


def grouped(**kw):
    return call("mma_gemm_grouped", dict(
        t=BF16, td=BF16, E=4, T=100, N=72, K=64, A=P, lda=64, B=P, ldb=64, sb=72 * 64, layout=0,
        at=R, C=0, ldc=0, D=Q, ldd=72), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(t=F32), UNSUP), (dict(td=F16), UNSUP), (dict(E=1025), UNSUP), (dict(E=-1), INVALID),
    (dict(layout=2), INVALID), (dict(T=-1), INVALID), (dict(at=0), INVALID), (dict(A=0), INVALID),
    (dict(B=0), INVALID), (dict(D=0), INVALID), (dict(lda=32), INVALID), (dict(ldb=32), INVALID),
    (dict(sb=71 * 64), INVALID), (dict(layout=1), INVALID), (dict(ldd=71), INVALID),
    (dict(C=Q, ldc=80), INVALID), (dict(at=R + 2), MISAL), (dict(A=P + 2), MISAL),
    (dict(lda=68), MISAL), (dict(sb=72 * 64 + 4), MISAL), (dict(D=Q + 1), MISAL),
    (dict(E=0, at=0), OK), (dict(T=0, A=0), OK),
])
def test_grouped(kw, code):
    assert grouped(**kw) == code


def wgrad(**kw):
    return call("mma_gemm_grouped_wgrad", dict(
        t=F16, td=F32, E=4, T=100, N=72, K=64, DY=P, lddy=72, X=P, ldx=64, at=R, C=0, ldc=0, sc=0,
        D=Q, ldd=64, sd=72 * 64), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(t=I8), UNSUP), (dict(td=BF16), UNSUP), (dict(E=2000), UNSUP), (dict(at=0), INVALID),
    (dict(DY=0), INVALID), (dict(X=0), INVALID), (dict(D=0), INVALID), (dict(lddy=64), INVALID),
    (dict(ldd=63), INVALID), (dict(sd=71 * 64), INVALID), (dict(C=P, ldc=64, sc=64), INVALID),
    (dict(C=Q, ldc=64, sc=73 * 64), INVALID), (dict(DY=P + 4), MISAL), (dict(ldx=68), MISAL),
    (dict(D=Q + 2), MISAL), (dict(E=0), OK), (dict(N=0, DY=0), OK), (dict(K=0), OK),
])
def test_wgrad(kw, code):
    assert wgrad(**kw) == code


def grouped_f8(**kw):
    return call("mma_gemm_grouped_f8", dict(
        ta=E4M3, tb=E4M3, td=BF16, E=4, T=100, N=72, K=128, A=P, lda=128, SA=R, sarow=1, sablk=100,
        B=P, ldb=128, sb=72 * 128, SB=R, rows=128, sbg=1, sbrow=1, sbblk=1, at=R, C=0, ldc=0, D=Q,
        ldd=72), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(ta=BF16), UNSUP), (dict(E=1025), UNSUP), (dict(at=0), INVALID), (dict(sbg=-1), INVALID),
    (dict(sb=128), INVALID), (dict(sb=72 * 128 + 8), MISAL), (dict(at=R + 1), MISAL),
    (dict(E=0, at=0), OK),
])
def test_grouped_f8(kw, code):
    assert grouped_f8(**kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="these addresses are fake")
def test_valid_calls_end_at_the_device():
    assert norm() == norm(R=0) == norm(Y=Q, ldy=256) == norm(H=0) == norm(H=P) == NODEV
    assert back() == back(M=0, DY=0, H=0, DX=0, ws=0, bytes=0) == back(DX=P) == NODEV
    assert quant() == quant(rows=128) == quant(trans=1, ldq=144) == quant(f8=E5M2) == NODEV
    assert f8() == f8(rows=1) == f8(K=0, A=0, B=0, SA=0, SB=0) == f8(C=Q, ldc=130) == NODEV
    assert f8(ldd=131, td=F32) == f8(sarow=2, sablk=1) == NODEV
    assert grouped() == grouped(layout=1, ldb=72, sb=64 * 72) == grouped(K=0, A=0, B=0) == NODEV
    assert wgrad() == wgrad(T=0, DY=0, X=0) == wgrad(C=Q, ldc=64, sc=72 * 64) == NODEV
    assert grouped_f8() == grouped_f8(rows=1) == NODEV


# ------------------------------------------------------------ Python binding

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


E = torch.float8_e4m3fn


@pytest.mark.parametrize("f,error", [
    (lambda: mma.rmsnorm_f8(t(2, 8, dtype=torch.int8), t(8)), TypeError),
    (lambda: mma.rmsnorm_f8(t(8), t(8)), ValueError),
    (lambda: mma.rmsnorm_f8(t(2, 8), t(8)), ValueError),                     # not on the GPU
    (lambda: mma.rmsnorm_backward(t(2, 8), t(2, 8, dtype=torch.int32), t(8)), TypeError),
    (lambda: mma.quantize_f8(t(2, 8, dtype=torch.float64)), TypeError),
    (lambda: mma.quantize_f8(t(2, 8, 4)), ValueError),
    (lambda: mma.gemm_f8(t(2, 8), t(2, 1), t(4, 8), t(4, 1)), TypeError),
    (lambda: mma.gemm_f8(t(2, 8, dtype=E), t(2, 1), t(4, 8, dtype=E), t(4, 1)), ValueError),
    (lambda: mma.gemm_grouped(t(2, 8, dtype=torch.float32), t(1, 4, 8), t(2)), TypeError),
    (lambda: mma.gemm_grouped(t(2, 8, 1), t(1, 4, 8), t(2)), ValueError),
    (lambda: mma.gemm_grouped_wgrad(t(2, 8), t(2, 4), t(2)), ValueError),
    (lambda: mma.gemm_grouped_f8(t(2, 8), t(2, 1), t(1, 4, 8), t(1, 1, 1), t(2)), TypeError),
])
def test_binding_refuses(f, error):
    with pytest.raises(error):
        f()
