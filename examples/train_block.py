"""Trains a stack of pre-norm blocks with the layer operators and the Dion3 step.

Each block adds W2 act(W1 norm(s)) to the residual stream s.  What the backward
pass needs of a block is kept in 8 bits: the norm's output (W1's input), the
pre-activation and the activation (W2's input), in half of the bytes of
16-bit copies.  The weight gradients go straight into the tensors that the step
reads.  The data are synthetic: the stream of a fixed random teacher.

    python examples/train_block.py [--steps 30] [--tokens 2048] [--width 512] [--hidden 2048] [--keep 16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalizing_optimizer_shape_gb300 as d3  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """Parameters, gradients and momenta of one block, and what it keeps of a batch."""

    def __init__(self, tokens: int, width: int, hidden: int, keep: int, gen: torch.Generator):
        def mat(n, m):
            return (torch.randn(n, m, generator=gen, device="cuda") * m ** -0.5).to(BF16)
        self.w1, self.w2 = mat(hidden, width), mat(width, hidden)
        self.g1, self.g2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.m1 = torch.zeros(hidden, width, device="cuda")
        self.m2 = torch.zeros(width, hidden, device="cuda")
        self.gain, self.dgain = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        self.b1, self.db1 = torch.zeros(hidden, device="cuda"), torch.zeros(hidden, device="cuda")
        new = lambda n: torch.empty(tokens, n, dtype=BF16, device="cuda")  # noqa: E731
        self.s, self.rstd = new(width), torch.empty(tokens, device="cuda")  # the stream at this block
        self.y, self.u, self.branch = new(width), new(hidden), new(width)
        self.eight = keep == 8
        if self.eight:
            self.y8, self.z, self.u8 = (d3.alloc_packed8(tokens, n) for n in (width, hidden, hidden))
        else:
            self.y8, self.z, self.u8 = None, new(hidden), None

    def forward(self, x, stream):
        """Adds x to the stream (None: x starts it) and leaves the block's branch in self.branch."""
        if stream is None:
            self.s.copy_(x)
            d3.rms_norm(self.s, self.gain, self.y, y8=self.y8, rstd=self.rstd)
        else:
            d3.rms_norm(x, self.gain, self.y, residual=stream, h=self.s, y8=self.y8, rstd=self.rstd)
        d3.linear(self.y, self.w1, self.u, bias=self.b1, act=d3.ACT_SILU, z=self.z, y8=self.u8)

    def finish(self, out=None):
        """The branch, or with `out` the stream after this block."""
        d3.linear(self.u, self.w2, self.branch if out is None else out, residual=None if out is None else self.s)
        return self.branch if out is None else out

    def backward(self, ds, du, dy, ws):
        """Gradients from that of the stream after the block; ds becomes that of the stream before it."""
        d3.linear_backward(ds, self.u8 if self.eight else self.u, self.w2, dx=du, dw=self.g2, ws=ws)
        d3.linear_backward(du, self.y8 if self.eight else self.y, self.w1, dx=dy, dw=self.g1, db=self.db1,
                           act=d3.ACT_SILU, z=self.z, ws=ws)
        d3.rms_norm_backward(dy, self.s, self.gain, self.rstd, ds, dh=ds, dw=self.dgain, ws=ws)


class Stack:
    def __init__(self, layers, tokens, width, hidden, keep, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(tokens, width, hidden, keep, gen) for _ in range(layers)]
        self.out = torch.empty(tokens, width, dtype=BF16, device="cuda")
        self.du = torch.empty(tokens, hidden, dtype=BF16, device="cuda")
        self.dy = torch.empty(tokens, width, dtype=BF16, device="cuda")
        self.ws = d3.alloc_workspace(max(
            d3.linear_backward_workspace_size(tokens, width, hidden, dtype=BF16),
            d3.linear_backward_workspace_size(tokens, hidden, width, dtype=BF16),
            d3.rms_norm_backward_workspace_size(tokens, width)))
        self.hp = d3.HParams(f=0.5, mu=0.95, lr=0.02)
        b = self.blocks
        self.groups = [d3.Group([x.w1 for x in b], [x.g1 for x in b], [x.m1 for x in b]),
                       d3.Group([x.w2 for x in b], [x.g2 for x in b], [x.m2 for x in b])]
        self.step_ws = d3.alloc_workspace(d3.workspace_size(self.groups, self.hp))

    def forward(self, x):
        stream = None
        for b in self.blocks:
            b.forward(x, stream)
            last = b is self.blocks[-1]
            x, stream = b.finish(self.out if last else None), b.s
        return self.out

    def backward(self, ds):
        for b in reversed(self.blocks):
            b.backward(ds, self.du, self.dy, self.ws)

    def step(self, lr=1e-2):
        d3.step(self.groups, self.hp, self.step_ws)
        for b in self.blocks:  # the vectors take plain gradient steps
            b.gain.sub_(b.dgain, alpha=lr)
            b.b1.sub_(b.db1, alpha=lr)


def train(steps=30, tokens=2048, width=512, hidden=2048, layers=2, keep=8, seed=0):
    """Losses of `steps` steps."""
    teacher = Stack(layers, tokens, width, hidden, 16, seed + 1000)
    model = Stack(layers, tokens, width, hidden, keep, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(BF16)
        diff = model.forward(x).float() - teacher.forward(x).float()
        losses.append(diff.square().mean())
        model.backward((diff * (2.0 / diff.numel())).to(BF16))
        model.step()
    d3.device_status()
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 30), ("tokens", 2048), ("width", 512), ("hidden", 2048), ("layers", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--keep", type=int, choices=(8, 16), default=8, help="bits of the kept activations")
    for i, loss in enumerate(train(**vars(ap.parse_args()))):
        print(f"step {i:3d}  loss {loss:.5f}")
