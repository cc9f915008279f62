"""Refusals of the products with low-rank adapters, without a GPU."""
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


def call(fn, args, kw):
    for k, v in kw.items():
        assert k in args, k
        args[k] = v
    return getattr(binding.load(), fn)(*args.values(), None)


def product(**kw):
    return call("mma_gemm_lora", dict(
        ti=BF16, td=BF16, T=100, N=256, K=128, rank=16, X=P, ldx=128, W=P, ldw=128, A=P, lda=128, sa=2048,
        B=P, ldb=16, sb=4096, layout=0, requests=5, off=P, of=P, total=3, sc=P, C=0, ldc=0, D=Q, ldd=256,
        S=R, lds=16, ws=R, bytes=1 << 20), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(ti=F32), UNSUP), (dict(td=F16), UNSUP), (dict(T=-1), INVALID), (dict(rank=-1), INVALID),
    (dict(rank=129, lds=136, ldb=136), UNSUP), (dict(requests=-1), INVALID), (dict(requests=65537), UNSUP),
    (dict(total=-1), INVALID), (dict(total=65536), UNSUP), (dict(layout=2), INVALID), (dict(off=0), INVALID),
    (dict(off=P + 2), MISAL), (dict(of=P + 1), MISAL), (dict(sc=P + 2), MISAL), (dict(X=0), INVALID),
    (dict(ldx=120), INVALID), (dict(ldx=132), MISAL), (dict(X=P + 2), MISAL), (dict(W=0), INVALID),
    (dict(ldw=64), INVALID), (dict(A=0), INVALID), (dict(A=P + 8), MISAL), (dict(lda=64), INVALID),
    (dict(sa=1000), INVALID), (dict(sa=2052), MISAL), (dict(B=0), INVALID), (dict(ldb=8), INVALID),
    (dict(ldb=20, sb=8192), MISAL), (dict(sb=4000), INVALID), (dict(D=0), INVALID), (dict(ldd=255), INVALID),
    (dict(D=Q + 1), MISAL), (dict(C=Q, ldc=512), INVALID), (dict(C=P, ldc=8), INVALID), (dict(S=0), INVALID),
    (dict(S=R + 4), MISAL), (dict(lds=20), MISAL), (dict(lds=8), INVALID), (dict(ws=0), INVALID),
    (dict(ws=R + 8), MISAL), (dict(bytes=100 * 256 * 4 - 1), INVALID), (dict(T=200, bytes=35 * 256 * 4 + 200 * 16 * 2 - 1), INVALID),
    (dict(T=0, X=0, D=0, off=0), OK),
])
def test_product(kw, code):
    assert product(**kw) == code


def wgrad(**kw):
    return call("mma_gemm_lora_wgrad", dict(
        ti=BF16, td=F32, T=100, N=256, K=128, rank=16, dY=P, lddy=256, X=P, ldx=128, S=P, lds=16, U=P, ldu=16,
        requests=5, off=P, of=P, total=3, dA=Q, ldda=128, sda=2048, dB=Q, lddb=16, sdb=4096, acc=0, ws=R,
        bytes=1 << 26), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(ti=E4M3), UNSUP), (dict(td=F16), UNSUP), (dict(N=-1), INVALID), (dict(rank=129), UNSUP),
    (dict(N=128 * 65535, lddy=128 * 65535), UNSUP), (dict(off=0), INVALID), (dict(dY=0), INVALID),
    (dict(X=0), INVALID), (dict(lddy=128), INVALID), (dict(ldx=130), MISAL), (dict(S=0), INVALID),
    (dict(U=0), INVALID), (dict(S=P + 2), MISAL), (dict(ldu=15), INVALID), (dict(lds=8), INVALID),
    (dict(dA=0), INVALID), (dict(dB=0), INVALID), (dict(ldda=64), INVALID), (dict(sda=100), INVALID),
    (dict(lddb=8), INVALID), (dict(dB=Q + 2), MISAL), (dict(ws=0), INVALID), (dict(bytes=1000), INVALID),
    (dict(ws=R + 4), MISAL), (dict(rank=0), OK), (dict(total=0), OK),
    (dict(requests=65537), UNSUP), (dict(requests=1025, total=1025, bytes=1 << 40), UNSUP), (dict(requests=1025, bytes=1 << 17), INVALID),
])
def test_wgrad(kw, code):
    assert wgrad(**kw) == code


def test_workspaces():
    f, g = binding.load().mma_gemm_lora_workspace, binding.load().mma_gemm_lora_wgrad_workspace
    assert f(BF16, BF16, 100, 30, 16, 3) == 12000 and f(BF16, F32, 200, 32, 17, 3) == 21 * 32 * 4 + 200 * 24 * 6
    assert f(F16, F32, 200, 32, 17, 3) == 21 * 32 * 4 + 200 * 24 * 4 and f(BF16, BF16, 10, 8, 0, 1) == 0
    assert g(BF16, F32, 0, 8, 8, 8, 3, 3) == 0 and g(BF16, F32, 1, 1, 1, 129, 1, 1) == 0
    assert g(BF16, F32, 100, 256, 128, 20, 5, 5) == 7 * 20 * 384 * 4 + 2 * 3 * 100 * 24 * 2
    assert g(F16, F16, 100, 256, 128, 20, 5, 5) == 7 * 20 * 384 * 4 + 2 * 100 * 24 * 2
    # rows in the order of their adapters: where that takes less, and with many requests
    few = g(F16, F16, 100, 256, 128, 20, 3, 3)
    assert g(F16, F16, 100, 256, 128, 20, 8, 3) == 10 * 20 * 384 * 4 + 2 * 100 * 24 * 2
    assert g(F16, F16, 100, 256, 128, 20, 9, 3) == few + (2 * 9 + 3 + 2 + 100 + 1) * 4 + 100 * 384 * 2
    assert f(BF16, BF16, 2000, 32, 16, 1025) == 2000 * 32 * 4


def test_binding():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 8, dtype=torch.bfloat16)
    at = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mma.gemm_lora(x, w, a, b, at)
    with pytest.raises(TypeError):
        mma.gemm_lora(x.float(), w, a, b, at)
    with pytest.raises(ValueError):
        mma.gemm_lora(x, w, a, b, at, b_layout="none")
