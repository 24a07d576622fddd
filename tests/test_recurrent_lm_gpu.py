"""The recurrent language model example: every language-model operator together
with the feed-forward ones and the optimizer step.  Its gradients against
torch's autograd in fp32 on the same bf16 parameters, with checkpoints in 8 bits
against without, and a few steps of training."""

import os
import sys

import numpy as np
import pytest

from gpu_helpers import require_gpu, torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(tokens=300, width=136, hidden=264, blocks=2, vocab=77)


@pytest.fixture(scope="module")
def example():
    require_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import recurrent_lm
    finally:
        sys.path.pop(0)
    return recurrent_lm


def rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def inputs(example, seed=5):
    gen = torch.Generator()
    gen.manual_seed(seed)
    ids, labels, starts = example.batch(SIZES["tokens"], SIZES["vocab"], 6, gen)
    ids[17] = -1                                        # padding
    return ids, labels, starts


def recurrence(x, g, starts):
    c, rows, h = torch.sigmoid(g), [], None
    first = set(starts.tolist())
    for t in range(len(x)):
        h = torch.zeros_like(x[0]) if t in first else h
        h = h + c[t] * (x[t] - h)
        rows.append(h)
    return torch.stack(rows)


def test_gradients_match_autograd(example):
    """Activations and their gradients are rounded to bf16 (2^-9 of their values on
    average) at nine places a block on the way forward and twelve back, and four
    places outside: sqrt(46) 2^-9 = 1.3e-2 over two blocks, times 3."""
    net = example.RecurrentLM(seed=3, **SIZES)
    ids, labels, starts = inputs(example)
    loss = net.loss_and_gradients(ids, labels, starts, 1.0)
    p = {id(q): q.model.float().requires_grad_() for q in net.parameters()}
    w = lambda q: p[id(q)]
    norm = lambda h, gamma: h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gamma
    known = (ids >= 0).float()[:, None]
    h = w(net.table)[ids.clamp(min=0)] * net.scale * known
    for b in net.blocks:
        n = norm(h, w(b.gamma1))
        x, g = n @ w(b.wx).t() + w(b.bx), n @ w(b.wg).t() + w(b.bg)
        h = recurrence(x, g, starts) @ w(b.wo).t() + h
        n = norm(h, w(b.gamma2))
        h = torch.nn.functional.gelu(n @ w(b.w1).t() + w(b.b1), approximate="tanh") @ w(b.w2).t() + h
    logits = norm(h, w(net.gamma)) @ w(net.head).t()
    want = torch.nn.functional.cross_entropy(logits, labels, ignore_index=-1, reduction="none")
    want.sum().backward()
    assert rel(loss, want) < 4e-2
    for q in net.parameters():
        assert rel(q.grad, w(q).grad) < 4e-2


def test_checkpoints_in_8_bits(example):
    """The forward pass is the same; a gradient differs by what e4m3 leaves of the
    pre-activation: z is off by 2^-4 of itself at most, gelu and its derivative
    by 1.13 times that, and |z| is 1.6 times gelu(z) and 1.2 times gelu'(z) in
    the mean square for normal z: 1.13 * 1.6 * 2^-4 = 0.11."""
    ids, labels, starts = inputs(example)
    nets = [example.RecurrentLM(seed=3, checkpoint=c, **SIZES) for c in (False, True)]
    losses = [n.loss_and_gradients(ids, labels, starts, 1.0) for n in nets]
    assert torch.equal(*losses)
    assert torch.equal(nets[0].head.grad, nets[1].head.grad)
    for a, b in zip(nets[0].parameters(), nets[1].parameters()):
        assert rel(b.grad, a.grad) < 0.11


@pytest.mark.parametrize("checkpoint", [False, True])
def test_training_runs(example, checkpoint):
    losses = example.train(steps=4, sequences=5, checkpoint=checkpoint, log=None, **SIZES)
    assert len(losses) == 4 and all(np.isfinite(losses))
