"""Refusals of the router and its gradient, without a GPU."""
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


def forward(**kw):
    return call("mma_route", dict(
        type=F32, T=1000, E=64, k=4, X=P, ldx=64, mask=0, norm=1, w=Q, ex=Q, order=Q, place=Q, off=Q,
        share=Q, loss=Q, tokens=Q, ws=R, bytes=1 << 24), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=I8), UNSUP), (dict(type=E4M3), UNSUP), (dict(T=-1), INVALID), (dict(E=0), INVALID),
    (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(E=1025, ldx=1025), UNSUP), (dict(k=33), UNSUP),
    (dict(T=1 << 29), UNSUP), (dict(X=0), INVALID), (dict(X=P + 2), MISAL), (dict(ldx=63), INVALID),
    (dict(w=0), INVALID), (dict(ex=0), INVALID), (dict(order=0), INVALID), (dict(place=0), INVALID),
    (dict(off=0), INVALID), (dict(share=0), INVALID), (dict(loss=0), INVALID), (dict(tokens=0), INVALID),
    (dict(off=Q + 2), MISAL), (dict(ws=0), INVALID), (dict(bytes=64), INVALID), (dict(ws=R + 1), MISAL),
    (dict(T=0, off=0), INVALID),
])
def test_forward(kw, code):
    assert forward(**kw) == code


def test_workspace():
    f = binding.load().mma_route_workspace
    assert f(0, 64) == 0 and f(96, 64) == 0 and f(32, 256) == 0 and f(-1, 64) == 0 and f(1000, 0) == 0
    assert f(97, 64) == (7 * (2 * 64 + 2) + 66) * 4 and f(33, 256) > 0
    assert f(10 ** 8, 64) <= (304 * (2 * 64 + 2) + 66) * 4


def back(**kw):
    return call("mma_route_backward", dict(
        type=F32, T=1000, E=64, k=4, X=P, ldx=64, mask=0, norm=1, w=P, ex=P, off=P, tokens=P, dw=P,
        dl=P, dx=Q, lddx=64), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(type=F64), UNSUP), (dict(k=65), INVALID), (dict(X=0), INVALID), (dict(dx=0), INVALID),
    (dict(lddx=8), INVALID), (dict(dx=P, lddx=128), INVALID), (dict(w=0), INVALID), (dict(ex=0), INVALID),
    (dict(off=0), INVALID), (dict(tokens=0), INVALID), (dict(dw=P + 2), MISAL), (dict(dl=P + 1), MISAL),
    (dict(dx=Q + 2), MISAL), (dict(T=0, X=0, dx=0), OK),
])
def test_backward(kw, code):
    assert back(**kw) == code


def test_binding():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        mma.route(x, 2)
    with pytest.raises(TypeError):
        mma.route(x.double(), 2)
    with pytest.raises(ValueError):
        mma.route(x[0], 2)
