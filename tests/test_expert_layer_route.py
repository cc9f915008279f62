"""The example layer's router where the GPU's is not used, against the definition.

Weights: FP32 exponentials and sums of at most 40 terms, below 2^-18 of the weight.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from mixed_precision_dense_02_gb300 import expert_layer


def by_loops(x, k):
    """The definition, a token at a time: of equal logits the lowest index."""
    choices = []
    for t, row in enumerate(x.double().tolist()):
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        top = max(row)
        w = [math.exp(row[e] - top) for e in best]
        choices += [(e, t, v / sum(w)) for e, v in zip(best, w)]
    at = sorted(range(len(choices)), key=lambda c: choices[c][0])
    offsets = [sum(c[0] < e for c in choices) for e in range(x.shape[1] + 1)]
    return at, [choices[c][1] for c in at], [choices[c][2] for c in at], offsets


def check(got, x, k):
    order, token, weight, offsets = by_loops(x, k)
    assert got[0].tolist() == order and got[1].tolist() == token and got[3].tolist() == offsets
    assert got[0].dtype == got[1].dtype == torch.int64 and got[3].dtype == torch.int32
    assert all(abs(a - b) <= 2.0 ** -18 * b for a, b in zip(got[2].tolist(), weight))


def logits(t, e, kind):
    g = torch.Generator().manual_seed(t + e)
    return (4 * torch.randn(t, e, generator=g)).round().div(2).to(kind)  # many equal ones


@pytest.mark.parametrize("t,e,k", [(1, 4, 1), (30, 8, 2), (7, 50, 40), (3, 1500, 5)])
@pytest.mark.parametrize("kind", [torch.float32, torch.float64, torch.bfloat16])
def test_route_on_the_cpu(t, e, k, kind):
    x = logits(t, e, kind)
    check(expert_layer.route(x, k), x, k)


def test_gradient_through_the_weights():
    x = logits(9, 6, torch.float32).requires_grad_()
    expert_layer.route(x, 2)[2].square().sum().backward()
    assert x.grad.abs().sum() > 0
