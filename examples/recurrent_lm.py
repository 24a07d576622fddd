"""Trains a small recurrent language model on synthetic token sequences of
different lengths, from the tokens to the optimizer step in the library's
operators:

    h = embedding[token] * sqrt(width)
    per block:  n = rmsnorm(h);  x = n wx^T + bx;  g = n wg^T + bg
                h = recurrence(x, g) wo^T + h
                n = rmsnorm(h);  h = gelu(n w1^T + b1) w2^T + h
    loss = cross_entropy(rmsnorm(h) head^T, next token)

    python examples/recurrent_lm.py [--steps 30] [--tokens 2048] [--width 256]
                                    [--hidden 1024] [--blocks 2] [--vocab 1000]
                                    [--sequences 8] [--checkpoint]

With --checkpoint a block keeps its pre-activation in 8 bits from the forward
to the backward pass, instead of that and the activation in bf16: 1.03 bytes
an element for 4.  The embedding and the head go to AdamW, the blocks' matrices
to Muon.  All buffers are allocated once; a step allocates nothing.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_optimizer_gb300 as mp

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def new(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Parameter:
    """fp32 master, gradient and optimizer state, and the bf16 model copy."""

    def __init__(self, value, embedding_or_output=False):
        self.main, self.grad = value.float().contiguous(), torch.zeros_like(value, dtype=FP32)
        self.m, self.v = torch.zeros_like(self.main), torch.zeros_like(self.main)
        self.model, self.end = self.main.to(BF16), embedding_or_output

    def entry(self):
        return mp.Param(self.main, self.grad, self.m, self.v, self.model, embedding_or_output=self.end)


class Block:
    def __init__(self, tokens, width, hidden, normal, checkpoint):
        one, zero = lambda n: Parameter(torch.ones(n, device="cuda")), lambda n: Parameter(torch.zeros(n, device="cuda"))
        square = lambda: Parameter(normal(width, width, std=width ** -0.5))
        self.gamma1, self.wx, self.bx, self.wg, self.bg, self.wo = one(width), square(), zero(width), square(), zero(width), square()
        self.gamma2, self.w1, self.b1 = one(width), Parameter(normal(hidden, width, std=width ** -0.5)), zero(hidden)
        self.w2 = Parameter(normal(width, hidden, std=hidden ** -0.5))
        self.h1, self.n1, self.r1 = None, new(tokens, width), new(tokens, dtype=FP32)      # h1: the stream as it came
        self.x, self.g, self.s = new(tokens, width), new(tokens, width), new(tokens, width)
        self.states = mp.recurrence_states(tokens, width, BF16)
        self.h2, self.n2, self.r2, self.out = new(tokens, width), new(tokens, width), new(tokens, dtype=FP32), new(tokens, width)
        self.checkpoint = checkpoint
        if checkpoint:
            self.q, self.scale = new(tokens, hidden, dtype=E4M3), new(tokens, -(-hidden // 32), dtype=torch.uint8)
        else:
            self.z, self.u = new(tokens, hidden), new(tokens, hidden)

    def parameters(self):
        return [self.gamma1, self.wx, self.bx, self.wg, self.bg, self.wo, self.gamma2, self.w1, self.b1, self.w2]

    def forward(self, h, starts, shared):
        ws = shared.ws
        self.h1 = h
        mp.rmsnorm(h, self.gamma1.model, y=self.n1, rstd=self.r1)
        mp.linear(self.n1, self.wx.model, self.x, bias=self.bx.model, workspace=ws)
        mp.linear(self.n1, self.wg.model, self.g, bias=self.bg.model, workspace=ws)
        mp.gated_recurrence(self.x, self.g, self.s, starts=starts, states=self.states)
        mp.linear(self.s, self.wo.model, self.h2, residual=h, workspace=ws)
        mp.rmsnorm(self.h2, self.gamma2.model, y=self.n2, rstd=self.r2)
        z, u = (shared.z, shared.u) if self.checkpoint else (self.z, self.u)
        mp.linear(self.n2, self.w1.model, u, bias=self.b1.model, act="gelu", z=z, workspace=ws)
        if self.checkpoint:
            mp.checkpoint_save(z, self.q, self.scale)
        mp.linear(u, self.w2.model, self.out, residual=self.h2, workspace=ws)
        return self.out

    def backward(self, dout, starts, shared):
        """dout: gradient of the block's output, in a buffer that it may write over
        with that of its input."""
        ws, norm_ws, w, t = shared.ws, shared.norm_ws, shared.dw, dict(accumulate=False)
        z, u = (shared.z, shared.u) if self.checkpoint else (self.z, self.u)
        if self.checkpoint:
            mp.checkpoint_restore(self.q, self.scale, z=z, y=u, act="gelu")
        mp.linear_backward(dout, u, self.w2.model, dx=shared.dz, z_prev=z, act_prev="gelu", dw=self.w2.grad, workspace=ws, **t)
        mp.linear_backward(shared.dz, self.n2, self.w1.model, dx=w[0], dw=self.w1.grad, dbias=self.b1.grad, workspace=ws, **t)
        mp.rmsnorm_backward(w[0], self.h2, self.gamma2.model, self.r2, dout, dh=dout, dgamma=self.gamma2.grad,
                            workspace=norm_ws, **t)
        mp.linear_backward(dout, self.s, self.wo.model, dx=w[0], dw=self.wo.grad, workspace=ws, **t)
        mp.gated_recurrence_backward(w[0], self.x, self.g, self.states, w[1], w[2], starts=starts)
        mp.linear_backward(w[1], self.n1, self.wx.model, dx=w[0], dw=self.wx.grad, dbias=self.bx.grad, workspace=ws, **t)
        mp.linear_backward(w[2], self.n1, self.wg.model, dx=w[1], dw=self.wg.grad, dbias=self.bg.grad, workspace=ws, **t)
        torch.add(w[0], w[1], out=w[0])
        mp.rmsnorm_backward(w[0], self.h1, self.gamma1.model, self.r1, dout, dh=dout, dgamma=self.gamma1.grad,
                            workspace=norm_ws, **t)


class Shared:
    """Buffers that the blocks use one after another."""

    def __init__(self, tokens, width, hidden, vocab, checkpoint):
        self.z, self.u = (new(tokens, hidden), new(tokens, hidden)) if checkpoint else (None, None)
        self.dz, self.dw = new(tokens, hidden), [new(tokens, width) for _ in range(3)]
        sizes = ((hidden, width), (width, hidden), (width, width), (vocab, width))
        self.ws = max((mp.linear_workspace(tokens, n, k, any_layout=True) for n, k in sizes), key=torch.numel)
        self.norm_ws = mp.rmsnorm_workspace(tokens, width)


class RecurrentLM:
    def __init__(self, tokens=2048, width=256, hidden=1024, blocks=2, vocab=1000, checkpoint=False, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        normal = lambda *s, std: torch.randn(*s, generator=gen, device="cuda") * std
        self.scale = math.sqrt(width)
        self.table = Parameter(normal(vocab, width, std=width ** -0.5), embedding_or_output=True)
        self.blocks = [Block(tokens, width, hidden, normal, checkpoint) for _ in range(blocks)]
        self.gamma = Parameter(torch.ones(width, device="cuda"))
        self.head = Parameter(normal(vocab, width, std=width ** -0.5), embedding_or_output=True)
        self.h0, self.n, self.rstd = new(tokens, width), new(tokens, width), new(tokens, dtype=FP32)
        self.logits, self.loss, self.dh = new(tokens, vocab), new(tokens, dtype=FP32), new(tokens, width)
        self.shared = Shared(tokens, width, hidden, vocab, checkpoint)
        self.embedding_ws = mp.embedding_workspace(tokens, vocab, width)
        self.params = mp.prepare([p.entry() for p in self.parameters()])
        self.opt_ws = mp.alloc_workspace(mp.workspace_size(self.params.params))
        self.step_no = 0

    def parameters(self):
        return [self.table, self.gamma, self.head] + [p for b in self.blocks for p in b.parameters()]

    def loss_and_gradients(self, tokens, labels, starts, scale):
        """The rows' losses; main_grad of every parameter for the sum of the losses
        times scale.  labels outside the vocabulary do not count."""
        mp.embedding(tokens, self.table.model, self.h0, scale=self.scale)
        h = self.h0
        for b in self.blocks:
            h = b.forward(h, starts, self.shared)
        mp.rmsnorm(h, self.gamma.model, y=self.n, rstd=self.rstd)
        ws = self.shared.ws
        mp.linear(self.n, self.head.model, self.logits, workspace=ws)
        mp.cross_entropy(self.logits, labels, self.loss, dlogits=self.logits, scale=scale)
        mp.linear_backward(self.logits, self.n, self.head.model, dx=self.shared.dw[0], dw=self.head.grad, accumulate=False,
                           workspace=ws)
        mp.rmsnorm_backward(self.shared.dw[0], h, self.gamma.model, self.rstd, self.dh, dgamma=self.gamma.grad, accumulate=False,
                            workspace=self.shared.norm_ws)
        for b in reversed(self.blocks):
            b.backward(self.dh, starts, self.shared)
        mp.embedding_backward(tokens, self.dh, self.table.grad, scale=self.scale, accumulate=False, workspace=self.embedding_ws)
        return self.loss

    def step(self, lr=0.01, adam_lr=2e-3):
        self.step_no += 1
        mp.mixed_step(self.params, mp.muon_hp(lr=lr), mp.adamw_hp(lr=adam_lr, weight_decay=0.0, step=self.step_no), self.opt_ws)


def batch(tokens, vocab, sequences, gen):
    """Packed sequences of random lengths, each from a random token on along a fixed
    walk through the vocabulary: (tokens, next tokens with -1 at each sequence's
    end, starts)."""
    cuts = torch.randint(0, tokens + 1, (sequences - 1,), generator=gen).sort().values.tolist()
    starts = [0] + cuts + [tokens]
    ids, labels = torch.empty(tokens, dtype=torch.int64), torch.empty(tokens, dtype=torch.int64)
    for a, b in zip(starts, starts[1:]):
        if b > a:
            first = int(torch.randint(0, vocab, (1,), generator=gen))
            ids[a:b] = (first + torch.arange(b - a) * 7) % vocab
            labels[a:b - 1], labels[b - 1] = ids[a + 1:b], -1
    return ids.cuda(), labels.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda")


def train(steps=30, tokens=2048, width=256, hidden=1024, blocks=2, vocab=1000, sequences=8, checkpoint=False, log=print):
    net = RecurrentLM(tokens, width, hidden, blocks, vocab, checkpoint)
    gen = torch.Generator()
    gen.manual_seed(1)
    losses = []
    for k in range(steps):
        ids, labels, starts = batch(tokens, vocab, sequences, gen)
        rows = net.loss_and_gradients(ids, labels, starts, 1.0)     # both optimizers are scale-free
        losses.append(float(rows.sum() / (labels >= 0).sum()))
        net.step()
        if log and (k % 5 == 0 or k == steps - 1):
            log(f"step {k:3d}  loss {losses[-1]:.4f}")
    assert mp.device_status(net.shared.ws) == mp.OPT_OK
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 30), ("tokens", 2048), ("width", 256), ("hidden", 1024), ("blocks", 2), ("vocab", 1000),
                        ("sequences", 8)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--checkpoint", action="store_true", help="pre-activations in 8 bits between the passes")
    train(**vars(ap.parse_args()))
