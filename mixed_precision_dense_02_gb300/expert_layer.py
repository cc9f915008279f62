"""A layer of experts on the 8-bit and grouped operators, as an example.

    python -m mixed_precision_dense_02_gb300.expert_layer

A residual stream is normalised, each token goes to its best two of a few
experts (two matrices with a gate between them), and what they return is
added up with the router's weights.  ``serve`` runs it on 8-bit operands:
norm with 8-bit output, grouped 8-bit products, quantiser in between.
``Trainer.step`` runs a step of training on 16-bit operands: grouped
products, their gradients for the inputs and the weights, and the norm's
gradient.  The command runs both on the GPU and prints how far they are from
the same formulas in 32 bits.
"""
from __future__ import annotations

import torch

from . import binding as mma

EPS = 1e-6


def route(logits, k):
    """The tokens of each expert: (order, token, weight, offsets).

    ``order`` sorts the k choices of every token by expert; ``token`` and
    ``weight`` are the sorted choices' tokens and router weights; expert e has
    the rows ``offsets[e]`` to ``offsets[e + 1]`` of them.
    """
    weight, expert = torch.topk(torch.softmax(logits.float(), -1), k)
    weight = weight / weight.sum(-1, keepdim=True)
    order = torch.argsort(expert.reshape(-1), stable=True)
    counts = torch.bincount(expert.reshape(-1), minlength=logits.shape[-1])
    offsets = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=logits.device)
    offsets[1:] = counts.cumsum(0)
    return order, order // k, weight.reshape(-1)[order], offsets


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

    def step(self, x, residual, d_out, rate, k=2):
        """One step of gradient descent for a loss whose gradient by the
        output is ``d_out``.  Returns (output, gradients): the gradients of
        x (and of the residual), the norm's weights, up and down."""
        w = self.w
        _, _, h, y = mma.rmsnorm_f8(x, w.norm, residual, eps=EPS, y=True)
        order, token, weight, offsets = route(mma.gemm(y, w.router), k)
        rows = y[token]
        a = mma.gemm_grouped(rows, w.up, offsets)
        with torch.enable_grad():
            leaf = a.detach().requires_grad_()
            m = gate(leaf)
        b = mma.gemm_grouped(m.detach(), w.down, offsets, out_dtype=torch.float32)
        out = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, b * weight[:, None])
        # backward (the router's choice is taken as given)
        db = (d_out[token].float() * weight[:, None]).to(x.dtype)
        d_down = mma.gemm_grouped_wgrad(db, m.detach(), offsets)
        dm = mma.gemm_grouped(db, w.down, offsets, b_layout="row")
        m.backward(dm)
        da = leaf.grad
        d_up = mma.gemm_grouped_wgrad(da, rows, offsets)
        d_rows = mma.gemm_grouped(da, w.up, offsets, b_layout="row", out_dtype=torch.float32)
        dy = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, d_rows)
        dx, d_norm = mma.rmsnorm_backward(dy.to(x.dtype), h, w.norm, eps=EPS)
        w.up = (w.up.float() - rate * d_up).bfloat16()
        w.down = (w.down.float() - rate * d_down).bfloat16()
        w.norm = (w.norm.float() - rate * d_norm).bfloat16()
        return out, {"x": dx, "norm": d_norm, "up": d_up, "down": d_down}


def reference(x, residual, w, k=2, norm=None, up=None, down=None):
    """The layer in 32 bits, with autograd's tensors where given; the router
    sees the same 16-bit rows as the kernels'."""
    norm = w.norm.float() if norm is None else norm
    up = w.up.float() if up is None else up
    down = w.down.float() if down is None else down
    h = x.float() + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * norm
    _, _, _, y16 = mma.rmsnorm_f8(x.detach().to(residual.dtype), w.norm, residual, eps=EPS,
                                  y=True)
    _, token, weight, offsets = route(mma.gemm(y16, w.router), k)
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
