"""Trains a stack of residual feed-forward blocks on a synthetic regression
task, with every operator of the library where it would be used:

    h_i = h_{i-1} + (block i-1's output);   n = rmsnorm(h_i) * gamma
    u = gelu(n w1^T + b1);                   out = u w2^T + b2

    python examples/residual_mlp.py [--steps 30] [--tokens 2048] [--width 512]
                                    [--hidden 2048] [--blocks 4] [--e4m3]

The forward pass reads the bf16 model copies (with --e4m3: both operands of
every product in 8 bits with a scale per row), the backward pass leaves fp32
gradients in main_grad, and mixed_step updates the fp32 masters (Muon for the
matrices, AdamW for the rest) and writes the next step's bf16 copies.  All
buffers are allocated once; a step allocates nothing.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_optimizer_gb300 as mp

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Parameter:
    """fp32 master, gradient and optimizer state, and the bf16 model copy."""

    def __init__(self, value):
        self.main, self.grad = value.float().contiguous(), torch.zeros_like(value, dtype=FP32)
        self.m, self.v = torch.zeros_like(self.main), torch.zeros_like(self.main)
        self.model = self.main.to(BF16)

    def entry(self):
        return mp.Param(self.main, self.grad, self.m, self.v, self.model)


class Block:
    def __init__(self, tokens, width, hidden, e4m3, gen):
        normal = lambda *s, std: torch.randn(*s, generator=gen, device="cuda") * std
        new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")
        self.gamma = Parameter(torch.ones(width, device="cuda"))
        self.w1, self.b1 = Parameter(normal(hidden, width, std=width ** -0.5)), Parameter(torch.zeros(hidden, device="cuda"))
        self.w2, self.b2 = Parameter(normal(width, hidden, std=hidden ** -0.5)), Parameter(torch.zeros(width, device="cuda"))
        # what the backward pass needs: the stream, its norm, the pre-activation and the activation
        self.h, self.n, self.rstd = new(tokens, width), new(tokens, width), new(tokens, dtype=FP32)
        self.z, self.u, self.out = new(tokens, hidden), new(tokens, hidden), new(tokens, width)
        self.dz, self.dn, self.dh = new(tokens, hidden), new(tokens, width), new(tokens, width)
        self.q = {}
        if e4m3:
            for name, rows, cols in (("n", tokens, width), ("u", tokens, hidden), ("w1", hidden, width), ("w2", width, hidden)):
                self.q[name] = (new(rows, cols, dtype=E4M3), new(rows, dtype=FP32))

    def parameters(self):
        return [self.gamma, self.w1, self.b1, self.w2, self.b2]

    def forward(self, x, residual, ws):
        """h = x + residual (x alone in the first block); out = the block's output."""
        q = self.q
        nq, ns = q.get("n", (None, None))
        mp.rmsnorm(x, self.gamma.model, residual=residual, h=self.h, y=self.n, q=nq, q_scale=ns, rstd=self.rstd)
        if q:
            mp.quantize_rows(self.w1.model, *q["w1"])
            mp.quantize_rows(self.w2.model, *q["w2"])
            mp.linear(nq, q["w1"][0], self.u, bias=self.b1.model, act="gelu", z=self.z, x_scale=ns, w_scale=q["w1"][1],
                      workspace=ws)
            mp.quantize_rows(self.u, *q["u"])
            mp.linear(q["u"][0], q["w2"][0], self.out, bias=self.b2.model, x_scale=q["u"][1], w_scale=q["w2"][1],
                      workspace=ws)
        else:
            mp.linear(self.n, self.w1.model, self.u, bias=self.b1.model, act="gelu", z=self.z, workspace=ws)
            mp.linear(self.u, self.w2.model, self.out, bias=self.b2.model, workspace=ws)

    def backward(self, dout, ws, norm_ws):
        """dout: gradient of h + out, which reaches both; leaves that of h in self.dh."""
        mp.linear_backward(dout, self.u, self.w2.model, dx=self.dz, z_prev=self.z, act_prev="gelu", dw=self.w2.grad,
                           dbias=self.b2.grad, accumulate=False, workspace=ws)
        mp.linear_backward(self.dz, self.n, self.w1.model, dx=self.dn, dw=self.w1.grad, dbias=self.b1.grad,
                           accumulate=False, workspace=ws)
        mp.rmsnorm_backward(self.dn, self.h, self.gamma.model, self.rstd, self.dh, dh=dout, dgamma=self.gamma.grad,
                            accumulate=False, workspace=norm_ws)


class ResidualMLP:
    def __init__(self, tokens=2048, width=512, hidden=2048, blocks=4, e4m3=False, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.blocks = [Block(tokens, width, hidden, e4m3, gen) for _ in range(blocks)]
        self.y = torch.empty(tokens, width, dtype=BF16, device="cuda")
        self.ws, self.norm_ws = mp.linear_workspace(tokens, hidden, width), mp.rmsnorm_workspace(tokens, width)
        # the second product of a block has the widths the other way round
        back = mp.linear_workspace(tokens, width, hidden)
        self.ws = back if back.numel() > self.ws.numel() else self.ws
        self.params = mp.prepare([p.entry() for b in self.blocks for p in b.parameters()])
        self.opt_ws = mp.alloc_workspace(mp.workspace_size(self.params.params))
        self.step_no = 0

    def forward(self, x):
        h, out = x, None
        for b in self.blocks:
            b.forward(h, out, self.ws)
            h, out = b.h, b.out
        torch.add(h, out, out=self.y)
        return self.y

    def backward(self, dy):
        for b in reversed(self.blocks):
            b.backward(dy, self.ws, self.norm_ws)
            dy = b.dh
        return dy

    def step(self, lr=0.005, adam_lr=1e-3):
        self.step_no += 1
        mp.mixed_step(self.params, mp.muon_hp(lr=lr), mp.adamw_hp(lr=adam_lr, weight_decay=0.0, step=self.step_no),
                      self.opt_ws)


def train(steps=30, tokens=2048, width=512, hidden=2048, blocks=4, e4m3=False, log=print):
    """Regression onto a fixed random two-layer map; returns the losses."""
    net = ResidualMLP(tokens, width, hidden, blocks, e4m3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    t1, t2 = (torch.randn(width, width, generator=gen, device="cuda") * width ** -0.5 for _ in range(2))
    losses = []
    for k in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(BF16)
        target = x.float() + torch.tanh(x.float() @ t1) @ t2
        err = net.forward(x).float() - target
        losses.append(float(err.square().mean()))
        net.backward((err * (2.0 / err.numel() * 1e3)).to(BF16))     # a scaled loss: both optimizers are scale-free
        net.step()
        if log and (k % 5 == 0 or k == steps - 1):
            log(f"step {k:3d}  loss {losses[-1]:.4f}")
    assert mp.device_status(net.ws) == mp.OPT_OK
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 30), ("tokens", 2048), ("width", 512), ("hidden", 2048), ("blocks", 4)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--e4m3", action="store_true", help="forward products in 8 bits")
    train(**vars(ap.parse_args()))
