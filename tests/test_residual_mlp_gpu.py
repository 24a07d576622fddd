"""The residual feed-forward example: the operators and the optimizer step
together.  Its gradients against torch's autograd in fp32 on the same bf16
parameters, and a short training run in bf16 and in 8 bits."""

import os
import sys

import numpy as np
import pytest

from gpu_helpers import require_gpu, torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import residual_mlp
    finally:
        sys.path.pop(0)
    return residual_mlp


def rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def test_gradients_match_autograd(example):
    """Activations and their gradients are rounded to bf16 (2^-9 of their
    values on average) at five places a block on the way forward and back:
    over three blocks sqrt(30) 2^-9 = 1.1e-2, times 3."""
    net = example.ResidualMLP(tokens=300, width=136, hidden=264, blocks=3, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(300, 136, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(300, 136, generator=g, device="cuda").to(torch.bfloat16)
    y = net.forward(x)
    dx = net.backward(dy)
    xs = x.float().requires_grad_()
    h, out, leaves = xs, None, []
    for b in net.blocks:
        p = [q.model.float().requires_grad_() for q in b.parameters()]
        leaves.append(p)
        h = h if out is None else h + out
        n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * p[0]
        out = torch.nn.functional.gelu(n @ p[1].t() + p[2], approximate="tanh") @ p[3].t() + p[4]
    want = h + out
    want.backward(dy.float())
    assert rel(y, want) < 3.3e-2 and rel(dx, xs.grad) < 3.3e-2
    for b, p in zip(net.blocks, leaves):
        for mine, ref in zip(b.parameters(), p):
            assert rel(mine.grad, ref.grad) < 3.3e-2


@pytest.mark.parametrize("e4m3", [False, True])
def test_training_reduces_the_loss(example, e4m3):
    losses = example.train(steps=25, tokens=512, width=256, hidden=512, blocks=2, e4m3=e4m3, log=None)
    assert all(np.isfinite(losses)) and np.mean(losses[-3:]) < 0.5 * losses[0], losses
