"""A layer of experts, trained with the grouped products and served in 8 bits.

Training: two grouped products forward; backward their input gradients (the same
call, weights read transposed) and weight gradients.  Serving: the trained
weights are brought to 8 bits once, a scale for each output channel, and each
step's tokens with a scale for each token.  The experts' row counts stay on the
GPU throughout.

    python examples/expert_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_gemm_amd as lib  # noqa: E402


class GroupedLinear(torch.autograd.Function):
    """Y[r] = X[r] @ W[e] for the rows r of every expert e; W is E x K x N."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return lib.gemm_grouped(x, w, offsets, x.new_empty(x.shape[0], w.shape[2]))

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = lib.gemm_grouped(dy, w, offsets, torch.empty_like(x), transpose_w=True)
        if ctx.needs_input_grad[1]:
            dw = lib.gemm_grouped_wgrad(x, dy, offsets, torch.empty_like(w))
        return dx, dw, None


def route(x, router, experts, top=2):
    """The rows' order by expert, their tokens and shares, and the offsets."""
    share, chosen = (x.float() @ router).softmax(1).topk(top, 1)
    share = share / share.sum(1, keepdim=True)
    order = chosen.flatten().argsort(stable=True)
    counts = torch.zeros(experts, dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, chosen.flatten(), torch.ones_like(chosen.flatten(), dtype=torch.int32))
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = counts.cumsum(0)
    return order // top, share.flatten()[order], offsets


class ExpertLayer:
    def __init__(self, width, hidden, experts, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.experts = experts
        self.router = torch.randn(width, experts, device="cuda", generator=g) * width ** -0.5
        self.up = (torch.randn(experts, width, hidden, device="cuda", generator=g) * width ** -0.5).to(dtype)
        self.down = (torch.randn(experts, hidden, width, device="cuda", generator=g) * hidden ** -0.5).to(dtype)
        self.up.requires_grad_(), self.down.requires_grad_()

    def __call__(self, x):
        token, share, offsets = route(x, self.router, self.experts)
        h = torch.nn.functional.silu(GroupedLinear.apply(x[token], self.up, offsets))
        y = GroupedLinear.apply(h, self.down, offsets)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, token, y.float() * share[:, None])

    def train_step(self, x, target, rate):
        loss = (self(x) - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for w in (self.up, self.down):
                w -= rate * w.grad
                w.grad = None
        return loss.detach()


class ServedLayer:
    """The layer with weights and activations in 8 bits."""

    def __init__(self, layer):
        self.router, self.experts = layer.router, layer.experts
        self.up, self.down = self._to_8_bits(layer.up), self._to_8_bits(layer.down)

    @staticmethod
    def _to_8_bits(w):
        """E x K x N weights as E x N x K integers with a scale for each channel."""
        rows = w.detach().transpose(1, 2).reshape(-1, w.shape[1])
        q = torch.empty(rows.shape, dtype=torch.int8, device=w.device)
        scale = torch.empty(rows.shape[0], device=w.device)
        lib.quantize_rows(rows, q, scale)
        return q.view(w.shape[0], w.shape[2], w.shape[1]), scale.view(w.shape[0], w.shape[2])

    @staticmethod
    def _product(x, weights, offsets):
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scale = torch.empty(x.shape[0], device=x.device)
        lib.quantize_rows(x, q, scale)
        w, channel = weights
        return lib.igemm(q, scale, w, channel, x.new_empty(x.shape[0], w.shape[1]), offsets=offsets)

    def __call__(self, x):
        token, share, offsets = route(x, self.router, self.experts)
        h = torch.nn.functional.silu(self._product(x[token], self.up, offsets))
        y = self._product(h, self.down, offsets)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, token, y.float() * share[:, None])


def main(width=512, hidden=1024, experts=8, tokens=2048, steps=30, rate=100.0):
    """Trains on a teacher's outputs; returns the first and last loss, and the
    served layer's error on a prompt and on single tokens relative to the
    trained layer's outputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    teacher, layer = ExpertLayer(width, hidden, experts, seed=2), ExpertLayer(width, hidden, experts, seed=3)
    layer.router = teacher.router
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
        with torch.no_grad():
            target = teacher(x)
        losses.append(layer.train_step(x, target, rate))
    served, errors = ServedLayer(layer), []
    with torch.no_grad():
        for n in (tokens, 1):
            x = torch.randn(n, width, device="cuda", generator=g).bfloat16()
            want = layer(x)
            errors.append(((served(x) - want).norm() / want.norm()).item())
    return losses[0].item(), losses[-1].item(), errors


if __name__ == "__main__":
    first, last, errors = main()
    print(f"loss {first:.4f} -> {last:.4f}; 8-bit serving off by {errors[0]:.2%} (prompt), {errors[1]:.2%} (one token)")
