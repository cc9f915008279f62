"""The new operators as they are used together: the example layer with a trained
router, and a block of layer norm, a projection with adapters, router and experts,
forward and backward, against autograd in 64 bits.

Tolerances, in the norm.  Every tensor between the operators is rounded to bfloat16,
2^-8 of it at most; the block has at most eight such places on any way, so 8 * 2^-8 =
0.032, and a gradient goes through the rounded forward tensors and as many of its own:
twice that.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def rnd(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def relative(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def softmax_weights(logits, experts, normalize=True):
    p = torch.softmax(logits, -1)
    w = p.gather(1, experts)
    return p, w / w.sum(-1, keepdim=True) if normalize else w


def balance_loss(p, experts, e, k):
    counts = torch.bincount(experts.reshape(-1), minlength=e).double()
    return e * (counts / experts.numel() * p.mean(0)).sum()


@pytest.mark.parametrize("tokens,experts,width,hidden,k", [(300, 8, 256, 192, 2), (64, 4, 128, 128, 1), (500, 20, 264, 136, 4)])
def test_trained_router(tokens, experts, width, hidden, k):
    from mixed_precision_dense_02_gb300 import expert_layer as el
    x, r, d = (rnd(i, tokens, width).to(BF16) for i in range(3))
    w = el.Weights(experts, width, hidden, seed=1)
    router = w.router.clone()
    _, _, _, y = mma.rmsnorm_f8(x, w.norm, r, eps=el.EPS, y=True)
    logits = mma.gemm(y, router)
    chosen = mma.route(logits, k).experts.long()
    leaf = router.double().requires_grad_()
    p, weight = softmax_weights(y.double() @ leaf.t(), chosen)
    out = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
    for j in range(k):
        up, down = w.up.double()[chosen[:, j]], w.down.double()[chosen[:, j]]
        h = torch.einsum("tw,thw->th", y.double(), up)
        a, b = h.chunk(2, -1)
        out = out + weight[:, j, None] * torch.einsum("th,twh->tw", torch.nn.functional.silu(a) * b, down)
    ((out * d.double()).sum() + 5.0 * balance_loss(p, chosen, experts, k)).backward()
    got, grads = el.Trainer(w).step(x, r, d, rate=1e-3, k=k, balance=5.0)
    assert relative(got, out.detach()) < 0.032
    assert relative(grads["router"], leaf.grad) < 0.064
    want = (router.float() - 1e-3 * grads["router"]).bfloat16()
    assert torch.equal(w.router, want)


def test_block():
    """h = x + r; y = layer norm of h; z = y W + adapters; the experts' outputs of z,
    chosen and weighted by a router, one matrix each; loss = <out, d> + 3 balance."""
    t, width, inner, e, k, rank = 330, 256, 320, 12, 3, 16
    offsets = torch.tensor([0, 150, 151, 152, 250, 330], dtype=torch.int32, device="cuda")
    adapters = torch.tensor([1, 0, -1, 2, 1], dtype=torch.int32, device="cuda")
    scales = torch.tensor([0.5, 1.5, 1.0], device="cuda")
    x, r, d = rnd(1, t, width).to(BF16), rnd(2, t, width).to(BF16), rnd(3, t, width).to(BF16)
    g, bias = (1 + 0.2 * rnd(4, width)).to(BF16), (0.2 * rnd(5, width)).to(BF16)
    w = (rnd(6, inner, width) / width ** 0.5).to(BF16)
    a, b = (rnd(7, 3, rank, width) / width ** 0.5).to(BF16), (rnd(8, 3, inner, rank) / rank ** 0.5).to(BF16)
    router, experts = (rnd(9, e, inner) / inner ** 0.5).to(BF16), (rnd(10, e, width, inner) / inner ** 0.5).to(BF16)

    # forward
    y, h = mma.layernorm(x, g, bias, r)
    z, s = mma.gemm_lora(y, w, a, b, offsets, adapters, scales, sums=True)
    logits = mma.gemm(z, router)
    routing = mma.route(logits, k)
    order = routing.order.long()
    rows = z[order // k]
    parts = mma.gemm_grouped(rows, experts, routing.offsets, out_dtype=torch.float32)
    place = routing.place.long()
    out = (parts[place] * routing.weights[..., None]).sum(1)
    # backward
    d_rows = (d[order // k].float() * routing.weights.reshape(-1)[order][:, None]).to(BF16)
    d_experts = mma.gemm_grouped_wgrad(d_rows, rows, routing.offsets)
    dz = mma.gemm_grouped(d_rows, experts, routing.offsets, b_layout="row", out_dtype=torch.float32)[place].sum(1)
    d_weights = (parts[place] * d[:, None].float()).sum(-1)
    d_logits = torch.zeros(t, 16, dtype=BF16, device="cuda")[:, :e]
    d_logits.copy_(mma.route_backward(logits, routing, d_weights, torch.tensor(3.0, device="cuda")))
    whole = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    d_router = mma.gemm_grouped_wgrad(d_logits, z, whole)[0]
    dz = (dz + mma.gemm_grouped(d_logits, router[None], whole, b_layout="row", out_dtype=torch.float32)).to(BF16)
    dy, u = mma.gemm_lora(dz, w, b, a, offsets, adapters, scales, b_layout="row", sums=True)
    da, db = mma.gemm_lora_wgrad(dz, y, s, u, offsets, adapters, adapters_total=3)
    dx, dg, dbias = mma.layernorm_backward(dy, h, g)

    # the same in 64 bits, with the kernels' choices
    leaves = [v.double().requires_grad_() for v in (x, g, bias, a, b, router, experts)]
    x6, g6, b6, a6, bb6, r6, e6 = leaves
    y6 = torch.nn.functional.layer_norm(x6 + r.double(), (width,), g6, b6, 1e-5)
    z6 = [y6 @ w.double().t()]
    at = offsets.tolist()
    extra = torch.zeros(t, inner, dtype=torch.float64, device="cuda")
    for (i, j), c in zip(zip(at, at[1:]), adapters.tolist()):
        if c >= 0:
            extra = extra + torch.nn.functional.pad(scales[c].double() * (y6[i:j] @ a6[c].t()) @ bb6[c].t(), (0, 0, i, t - j))
    z6 = z6[0] + extra
    chosen = routing.experts.long()
    p, weight = softmax_weights(z6 @ r6.t(), chosen)
    out6 = sum(weight[:, j, None] * torch.einsum("ti,twi->tw", z6, e6[chosen[:, j]]) for j in range(k))
    ((out6 * d.double()).sum() + 3.0 * balance_loss(p, chosen, e, k)).backward()
    assert relative(out, out6.detach()) < 0.032
    for name, got, leaf in (("x", dx, x6), ("norm", dg, g6), ("bias", dbias, b6), ("adapters' A", da, a6), ("adapters' B", db, bb6),
                            ("router", d_router, r6), ("experts", d_experts, e6)):
        assert relative(got, leaf.grad) < 0.064, name


def test_layer_norm_in_8_bits_before_a_product():
    """Within 2^-4 per 8-bit value, uniformly spread, as the norm of the products'
    errors: 2 * 2^-5 of both operands'."""
    t, width, n = 200, 512, 264
    x, w = rnd(1, t, width).to(BF16), rnd(2, n, width) / width ** 0.5
    g, b = (1 + 0.2 * rnd(3, width)).to(BF16), (0.2 * rnd(4, width)).to(BF16)
    q, s, _ = mma.layernorm_f8(x, g, b)
    wq, ws = mma.quantize_f8(w, block_rows=128)
    got = mma.gemm_f8(q, s, wq, ws)
    want = torch.nn.functional.layer_norm(x.double(), (width,), g.double(), b.double(), 1e-5) @ w.double().t()
    assert relative(got, want) < 0.0625
