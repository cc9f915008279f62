"""Sizes of the products with low-rank adapters at which counters of 32 bits would run over,
without a GPU: the kernels' loops go on by up to 8 blocks of 1024 columns past the end."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from test_lora_refusals import UNSUP, lib, product, wgrad  # noqa: F401

MOST = 2 ** 31 - 2 ** 16
NEAR = [2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 31 - 1025, 2 ** 31 - 8192, MOST + 1]


@pytest.mark.parametrize("n", NEAR)
def test_refused(n):
    wide = dict(bytes=1 << 62)
    ld = -(-n // 8) * 8
    assert product(N=n, sb=16 * ld, ldd=ld, **wide) == UNSUP
    assert product(T=n, **wide) == UNSUP
    assert product(K=n, ldx=ld, ldw=ld, lda=ld, sa=16 * ld, **wide) == UNSUP
    assert wgrad(T=n, **wide) == UNSUP


def test_taken():
    """(as far as a call without a device goes)"""
    wide = dict(bytes=1 << 62)
    assert product(N=MOST, sb=16 * MOST, ldd=MOST, **wide) != UNSUP
    assert product(T=MOST, **wide) != UNSUP
    assert product(K=MOST, ldx=MOST, ldw=MOST, lda=MOST, sa=16 * MOST, **wide) != UNSUP
