"""The example's layer of experts: its gradients against plain torch in 64 bits,
and a short run from training to 8-bit serving."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def test_gradients():
    g = torch.Generator(device="cuda").manual_seed(0)
    off = torch.tensor([0, 5, 5, 40, 47], dtype=torch.int32, device="cuda")
    x = torch.randn(47, 24, device="cuda", generator=g).requires_grad_()
    w = torch.randn(4, 24, 20, device="cuda", generator=g).requires_grad_()
    dy = torch.randn(47, 20, device="cuda", generator=g)
    y = expert_layer.GroupedLinear.apply(x, w, off)
    y.backward(dy)
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    at = off.tolist()
    yd = torch.cat([xd[at[e]:at[e + 1]] @ wd[e] for e in range(4)])
    yd.backward(dy.double())
    # K roundings of 2^-23 of sums of K terms of size up to about 4 x 4 each.
    for got, want, steps in ((y, yd, 24), (x.grad, xd.grad, 20), (w.grad, wd.grad, 35)):
        assert (got.double() - want).abs().max() <= steps * steps * 16 * 2.0 ** -23


def test_training_then_serving():
    first, last, errors = expert_layer.main(width=256, hidden=512, tokens=1024, steps=20)
    assert last < 0.9 * first
    # Codes are off by half a step of 1/127 of a row's largest value, some 3 to 4
    # deviations: each of four quantised operands adds about 0.3 * 4 / 127 = 1 %.
    assert max(errors) < 0.05
