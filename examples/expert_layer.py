"""A norm and a layer of experts, trained with the grouped products and served in 8
or 4 bits.

Training: the norm and two grouped products forward; backward the norm's gradient,
the products' input gradients (the same call, weights read transposed) and weight
gradients.  Serving: the trained weights are brought to 8 bits once, a scale for each
output channel, or to microscaled 4-bit floats.  A prompt's tokens go from the norm
straight to codes with a scale each, and are multiplied sorted by expert; a decoding
step's few tokens go through the whole layer in one call.  The experts' row counts
stay on the GPU throughout.

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


class Norm(torch.autograd.Function):
    """x / sqrt(mean(x ** 2) + 1e-6) * weight, row by row."""

    @staticmethod
    def forward(ctx, x, weight):
        ctx.save_for_backward(x, weight)
        return lib.rms_norm(x, weight, torch.empty_like(x))

    @staticmethod
    def backward(ctx, dy):
        x, weight = ctx.saved_tensors
        return lib.rms_norm_grad(dy.contiguous(), x, weight, torch.empty_like(x), torch.empty_like(weight))


def choose(x, router, top=2):
    """Each token's experts and their shares."""
    share, chosen = (x.float() @ router).softmax(1).topk(top, 1)
    return share / share.sum(1, keepdim=True), chosen


def route(x, router, experts, top=2):
    """The rows' order by expert, their tokens and shares, and the offsets."""
    share, chosen = choose(x, router, top)
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
        self.norm = torch.ones(width, device="cuda", requires_grad=True)
        self.router = torch.randn(width, experts, device="cuda", generator=g) * width ** -0.5
        self.up = (torch.randn(experts, width, hidden, device="cuda", generator=g) * width ** -0.5).to(dtype)
        self.down = (torch.randn(experts, hidden, width, device="cuda", generator=g) * hidden ** -0.5).to(dtype)
        self.up.requires_grad_(), self.down.requires_grad_()

    def __call__(self, x):
        x = Norm.apply(x, self.norm)
        token, share, offsets = route(x, self.router, self.experts)
        h = torch.nn.functional.silu(GroupedLinear.apply(x[token], self.up, offsets))
        y = GroupedLinear.apply(h, self.down, offsets)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, token, y.float() * share[:, None])

    def train_step(self, x, target, rate):
        loss = (self(x) - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for w in (self.up, self.down, self.norm):
                w -= rate * w.grad
                w.grad = None
        return loss.detach()


class ServedLayer:
    """The layer with weights in 8 or 4 bits; a prompt's activations in as many."""

    FEW = 64  # tokens that one call takes through the whole layer

    def __init__(self, layer, bits=8):
        self.router, self.experts, self.bits = layer.router, layer.experts, bits
        self.norm = layer.norm.detach()
        self.up, self.down = self._narrow(layer.up), self._narrow(layer.down)

    def _narrow(self, w):
        """E x K x N weights as E x N x K codes, with a scale for each channel, or for
        each 32 values of one."""
        E, K, N = w.shape
        q, scale = self._codes(w.detach().transpose(1, 2).reshape(E * N, K))
        return q.view(E, N, -1), scale.view(E, N) if self.bits == 8 else scale.view(E, N, -1)

    def _codes(self, rows):
        M, K = rows.shape
        if self.bits == 8:
            return lib.quantize_rows(rows, torch.empty(M, K, dtype=torch.int8, device=rows.device),
                                     torch.empty(M, device=rows.device))
        return lib.quantize_mx4(rows, torch.empty(M, (K + 1) // 2, dtype=torch.uint8, device=rows.device),
                                torch.empty(M, (K + 31) // 32, dtype=torch.uint8, device=rows.device))

    def _product(self, codes, weights, offsets, dtype):
        (q, scale), (w, channel) = codes, weights
        multiply = lib.igemm if self.bits == 8 else lib.gemm_mx4
        return multiply(q, scale, w, channel, q.new_empty(q.shape[0], w.shape[1], dtype=dtype), offsets=offsets)

    def __call__(self, x):
        if x.shape[0] <= self.FEW:
            n = lib.rms_norm(x, self.norm, torch.empty_like(x))
            share, chosen = choose(n, self.router)
            y = x.new_empty(x.shape, dtype=torch.float32)
            return lib.expert_layer(n, chosen.int(), share, self.up[0], self.down[0], y, self.up[1], self.down[1],
                                    gated=False)
        n = torch.empty_like(x)
        if self.bits == 8:  # the norm's codes come with it
            codes = (torch.empty(x.shape, dtype=torch.int8, device=x.device), torch.empty(x.shape[0], device=x.device))
            lib.rms_norm(x, self.norm, n, Q=codes[0], scale=codes[1])
        else:
            codes = self._codes(lib.rms_norm(x, self.norm, n))
        token, share, offsets = route(n, self.router, self.experts)
        h = torch.nn.functional.silu(self._product([c[token] for c in codes], self.up, offsets, x.dtype))
        y = self._product(self._codes(h), self.down, offsets, x.dtype)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, token, y.float() * share[:, None])


def main(width=512, hidden=1024, experts=8, tokens=2048, steps=30, rate=100.0, bits=8):
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
    served, errors = ServedLayer(layer, bits), []
    with torch.no_grad():
        for n in (tokens, 1):
            x = torch.randn(n, width, device="cuda", generator=g).bfloat16()
            want = layer(x)
            errors.append(((served(x) - want).norm() / want.norm()).item())
    return losses[0].item(), losses[-1].item(), errors


if __name__ == "__main__":
    first, last, errors = main()
    print(f"loss {first:.4f} -> {last:.4f}; 8-bit serving off by {errors[0]:.2%} (prompt), {errors[1]:.2%} (one token)")
