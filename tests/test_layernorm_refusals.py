"""Refusals of the layer norm and its gradient, without a GPU."""
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


def norm(**kw):
    return call("mma_layernorm", dict(
        type=BF16, wt=BF16, M=4, N=256, X=P, ldx=256, R=P, ldr=256, W=P, B=P, eps=1e-6, pow2=0,
        H=Q, ldh=256, Y=0, ldy=0, Q=R, ldq=256, S=R, srow=1, sblk=4), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=I8), UNSUP), (dict(wt=F16), UNSUP), (dict(M=-1), INVALID), (dict(N=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(X=0), INVALID),
    (dict(W=0), INVALID), (dict(ldx=255), INVALID), (dict(ldr=8), INVALID), (dict(S=0), INVALID),
    (dict(Q=0, Y=0), INVALID), (dict(H=P, ldh=512), INVALID), (dict(B=P + 2), MISAL),
    (dict(X=P + 8), MISAL), (dict(ldx=257), MISAL), (dict(Y=Q, ldy=260), MISAL),
    (dict(M=0, X=0, Q=0, W=0), OK), (dict(N=0, X=0), OK),
])
def test_norm(kw, code):
    assert norm(**kw) == code


def back(**kw):
    return call("mma_layernorm_backward", dict(
        type=BF16, wt=F32, M=4, N=256, DY=P, lddy=256, H=P, ldh=256, W=P, eps=1e-6, R=0, ldr=0,
        DX=Q, lddx=256, DW=R, DB=R, ws=R, bytes=1 << 20), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=E4M3), UNSUP), (dict(wt=F16), UNSUP), (dict(M=-2), INVALID), (dict(DY=0), INVALID),
    (dict(H=0), INVALID), (dict(DX=0), INVALID), (dict(DW=0), INVALID), (dict(DB=0), INVALID),
    (dict(ws=0), INVALID), (dict(bytes=8 * 256 * 4 - 1), INVALID), (dict(DX=P, lddx=512), INVALID),
    (dict(DB=R + 2), MISAL), (dict(H=P + 4), MISAL), (dict(N=0), OK),
])
def test_backward(kw, code):
    assert back(**kw) == code


def test_workspace():
    f = binding.load().mma_layernorm_backward_workspace
    assert f(0, 4096) == 0 and f(4, 256) == 8 * 256 * 4
    assert f(10 ** 6, 256) == 2432 * 256 * 4 and f(10 ** 6, 4096) == 912 * 4096 * 4
    assert f(10 ** 6, 16384) == 912 * 16384 * 4 + 16 * 10 ** 6 and f(-1, 5) == 0


def test_binding():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mma.layernorm(x, w)
    with pytest.raises(TypeError):
        mma.layernorm(x.to(torch.int32), w)
    with pytest.raises(ValueError):
        mma.layernorm(x[0], w)
