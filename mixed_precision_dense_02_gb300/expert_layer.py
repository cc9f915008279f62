"""A layer of experts on the 8-bit and grouped operators, as an example.

    python -m mixed_precision_dense_02_gb300.expert_layer

A residual stream is normalised, each token goes to its best two of a few
experts (two matrices with a gate between them), and what they return is
added up with the router's weights.  ``serve`` runs it on 8-bit operands:
norm with 8-bit output, grouped 8-bit products, quantiser in between.
``Trainer.step`` runs a step of training on 16-bit operands: grouped
products, their gradients for the inputs and the weights, the norm's
gradient and, where asked for, the router's, with its balance loss.  The
command runs both on the GPU and prints how far they are from the same
formulas in 32 bits.
"""
from __future__ import annotations

import torch

from . import binding as mma

EPS = 1e-6


def route(logits, k):
    """The tokens of each expert: (order, token, weight, offsets).

    ``order`` sorts the k choices of every token by expert; ``token`` and
    ``weight`` are the sorted choices' tokens and router weights; expert e has
    the rows ``offsets[e]`` to ``offsets[e + 1]`` of them.  Logits that the GPU's
    router does not take (on the CPU, of other types, more than 1024 experts or 32
    choices, or with a gradient to be taken through the weights) go through torch.
    """
    if (logits.is_cuda and logits.dim() == 2 and not logits.requires_grad
            and logits.dtype in (torch.float32, torch.float16, torch.bfloat16)
            and logits.shape[1] <= 1024 and 1 <= k <= 32):
        return _sorted(mma.route(logits.contiguous(), k), k)
    return plain_route(logits, k)


def plain_route(logits, k):
    """``route`` in torch operations, of equal logits the lowest expert first."""
    if not 0 <= k <= logits.shape[-1]:
        raise ValueError(f"k must be at most {logits.shape[-1]}, not {k}")
    weight = torch.softmax(logits.float(), -1)
    expert = torch.sort(logits, dim=-1, descending=True, stable=True).indices[..., :k]
    weight = weight.gather(-1, expert)
    weight = weight / weight.sum(-1, keepdim=True)
    order = torch.argsort(expert.reshape(-1), stable=True)
    counts = torch.bincount(expert.reshape(-1), minlength=logits.shape[-1])
    offsets = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=logits.device)
    offsets[1:] = counts.cumsum(0)
    return order, order // k, weight.reshape(-1)[order], offsets


def _sorted(r, k):
    order = r.order.long()
    return order, order // k, r.weights.reshape(-1)[order], r.offsets


def gate(h):
    """silu(a) * b of the two halves of h's columns."""
    a, b = h.chunk(2, -1)
    return torch.nn.functional.silu(a) * b


class Weights:
    """A router (experts x width) and the experts' matrices: up (experts x
    2 * hidden x width), down (experts x width x hidden)."""

    def __init__(self, experts, width, hidden, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.norm = (1 + 0.1 * r(width)).bfloat16()
        self.router = (r(experts, width) / width ** 0.5).bfloat16()
        self.up = (r(experts, 2 * hidden, width) / width ** 0.5).bfloat16()
        self.down = (r(experts, width, hidden) / hidden ** 0.5).bfloat16()

    def in_8_bits(self):
        """up and down as 8-bit values with a scale per 128 x 128 block."""
        def each(w):
            # rows that start on 16-byte boundaries, as the products read them
            experts, rows, columns = w.shape
            q = torch.empty(experts, rows, -(-columns // 16) * 16, dtype=torch.uint8,
                            device=w.device)[..., :columns]
            scales = []
            for e in range(experts):
                m, s = mma.quantize_f8(w[e], block_rows=128)
                q[e] = m.view(torch.uint8)
                scales.append(s)
            return q.view(m.dtype), torch.stack(scales)
        return each(self.up), each(self.down)


def serve(x, residual, w, w8, k=2):
    """The layer on 8-bit operands; returns (output, new residual)."""
    (up, up_s), (down, down_s) = w8
    q, s, h, y = mma.rmsnorm_f8(x, w.norm, residual, eps=EPS, y=True)
    _, token, weight, offsets = route(mma.gemm(y, w.router), k)
    a = mma.gemm_grouped_f8(q.view(torch.uint8)[token].view(q.dtype), s[token], up, up_s, offsets)
    aq, as_ = mma.quantize_f8(gate(a))
    b = mma.gemm_grouped_f8(aq, as_, down, down_s, offsets, out_dtype=torch.float32)
    out = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, b * weight[:, None])
    return out.to(x.dtype), h


class Trainer:
    """Training of up and down on 16-bit operands, with 32-bit gradients."""

    def __init__(self, w):
        self.w = w

    def step(self, x, residual, d_out, rate, k=2, balance=None):
        """One step of gradient descent for a loss whose gradient by the
        output is ``d_out``.  Returns (output, gradients): the gradients of
        x (and of the residual), the norm's weights, up and down.  With
        ``balance`` the router is trained too: by its weights, and by
        ``balance`` times its balance loss (gradients: "router" as well).
        """
        w = self.w
        _, _, h, y = mma.rmsnorm_f8(x, w.norm, residual, eps=EPS, y=True)
        logits = mma.gemm(y, w.router)
        routing = mma.route(logits, k)
        order, token, weight, offsets = _sorted(routing, k)
        rows = y[token]
        a = mma.gemm_grouped(rows, w.up, offsets)
        with torch.enable_grad():
            leaf = a.detach().requires_grad_()
            m = gate(leaf)
        b = mma.gemm_grouped(m.detach(), w.down, offsets, out_dtype=torch.float32)
        out = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, b * weight[:, None])
        # backward (the router's choice is taken as given, and its weights too
        # unless it is trained)
        db = (d_out[token].float() * weight[:, None]).to(x.dtype)
        d_down = mma.gemm_grouped_wgrad(db, m.detach(), offsets)
        dm = mma.gemm_grouped(db, w.down, offsets, b_layout="row")
        m.backward(dm)
        da = leaf.grad
        d_up = mma.gemm_grouped_wgrad(da, rows, offsets)
        d_rows = mma.gemm_grouped(da, w.up, offsets, b_layout="row", out_dtype=torch.float32)
        dy = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, d_rows)
        d_router = None
        if balance is not None:
            place = routing.place.long()
            d_weight = (b[place] * d_out[:, None].float()).sum(-1)
            d_loss = torch.full((), balance, dtype=torch.float32, device=x.device)
            # (rows that start on 16-byte boundaries, as the products read them)
            experts = logits.shape[1]
            d_logits = torch.zeros(x.shape[0], -(-experts // 8) * 8, dtype=x.dtype,
                                   device=x.device)[:, :experts]
            d_logits.copy_(mma.route_backward(logits, routing, d_weight, d_loss))
            whole = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=x.device)
            d_router = mma.gemm_grouped_wgrad(d_logits, y, whole)[0]
            dy += mma.gemm_grouped(d_logits, w.router[None], whole, b_layout="row",
                                   out_dtype=torch.float32)
        dx, d_norm = mma.rmsnorm_backward(dy.to(x.dtype), h, w.norm, eps=EPS)
        w.up = (w.up.float() - rate * d_up).bfloat16()
        w.down = (w.down.float() - rate * d_down).bfloat16()
        w.norm = (w.norm.float() - rate * d_norm).bfloat16()
        grads = {"x": dx, "norm": d_norm, "up": d_up, "down": d_down}
        if d_router is not None:
            w.router = (w.router.float() - rate * d_router).bfloat16()
            grads["router"] = d_router
        return out, grads


def reference(x, residual, w, k=2, norm=None, up=None, down=None):
    """The layer in 32 bits and torch operations, with autograd's tensors where given;
    the router sees the same logits of 16-bit rows as the kernels'."""
    norm = w.norm.float() if norm is None else norm
    up = w.up.float() if up is None else up
    down = w.down.float() if down is None else down
    h = x.float() + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * norm
    _, _, _, y16 = mma.rmsnorm_f8(x.detach().to(residual.dtype), w.norm, residual, eps=EPS,
                                  y=True)
    _, token, weight, offsets = plain_route(mma.gemm(y16, w.router), k)
    at = offsets.tolist()
    parts = [gate(y[token[i:j]] @ up[e].t()) @ down[e].t()
             for e, (i, j) in enumerate(zip(at, at[1:]))]
    b = torch.cat(parts) * weight[:, None]
    return torch.zeros_like(h).index_add(0, token, b)


def relative(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def demo(tokens=1000, experts=8, width=512, hidden=768, seed=0):
    """Both paths on random data: the relative errors of their outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, r, d = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = Weights(experts, width, hidden, seed)
    out, _ = serve(x, r, w, w.in_8_bits())
    errors = {"served output": relative(out, reference(x, r, w))}
    xs = x.float().requires_grad_()
    p = [t.float().requires_grad_() for t in (w.norm, w.up, w.down)]
    want = reference(xs, r, w, norm=p[0], up=p[1], down=p[2])
    want.backward(d.float())
    out, grads = Trainer(w).step(x, r, d, rate=1e-3)
    errors["output"] = relative(out, want.detach())
    for name, t in zip(("x", "norm", "up", "down"), (xs, *p)):
        errors["gradient of " + name] = relative(grads[name], t.grad)
    mma.device_status()
    return errors


if __name__ == "__main__":
    for name, e in demo().items():
        print(f"{name:20s} relative error {e:.2e}")
