"""Trains a small recurrent language model with the framework's operators alone.

Token embedding; blocks of RMS norm, one matrix to gates and inputs, a gated
recurrence along the tokens of packed sequences and a matrix back onto the
residual stream; a norm and the head; log probabilities of the next tokens and
their gradient in the logits' place; all gradients clipped to a norm; the Dion3
step for the blocks' matrices.  Then it continues a few prompts token by token
with the recurrent states carried along.  The data are synthetic: sequences that
count upwards from a random start with a random stride.

    python examples/train_lm.py [--steps 60] [--tokens 2048] [--vocab 512] [--width 256] [--layers 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalizing_optimizer_shape_gb300 as d3  # noqa: E402

BF16 = torch.bfloat16
PAD = -1  # of ids and targets: no token


def new(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Block:
    """Parameters of one block, their gradients and momenta, and what a batch leaves in it."""

    def __init__(self, tokens: int, width: int, gen: torch.Generator):
        def mat(n, m):
            return (torch.randn(n, m, generator=gen, device="cuda") * m ** -0.5).to(BF16)
        self.w_in, self.w_out = mat(2 * width, width), mat(width, width)
        self.b_in = torch.zeros(2 * width, device="cuda")
        self.b_in[:width] = 2.0  # gates that remember
        self.gain = torch.ones(width, device="cuda")
        self.params = [self.w_in, self.w_out, self.b_in, self.gain]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.m_in, self.m_out = (torch.zeros(w.shape, device="cuda") for w in (self.w_in, self.w_out))
        self.s, self.y, self.h, self.branch = (new(tokens, width) for _ in range(4))
        self.u = new(tokens, 2 * width)  # gates | inputs
        self.rstd = new(tokens, dtype=torch.float32)
        self.width = width

    def forward(self, x, stream, offsets, first=None, last=None):
        """Adds x to the stream (None: x starts it) and returns the branch that follows."""
        if stream is None:
            self.s.copy_(x)
            d3.rms_norm(self.s, self.gain, self.y, rstd=self.rstd)
        else:
            d3.rms_norm(x, self.gain, self.y, residual=stream, h=self.s, rstd=self.rstd)
        d3.linear(self.y, self.w_in, self.u, bias=self.b_in)
        d3.recurrence(self.u[:, :self.width], self.u[:, self.width:], self.h, offsets=offsets, first=first, last=last)
        d3.linear(self.h, self.w_out, self.branch)
        return self.branch

    def backward(self, ds, offsets, tmp, ws):
        """Gradients from that of the stream after the block; ds becomes that before it."""
        dh, du, w = tmp.dh, tmp.du, self.width
        g_in, g_out, db, dgain = self.grads
        d3.linear_backward(ds, self.h, self.w_out, dx=dh, dw=g_out, ws=ws)
        d3.recurrence_backward(dh, self.u[:, :w], self.u[:, w:], self.h, du[:, :w], du[:, w:], offsets=offsets)
        d3.linear_backward(du, self.y, self.w_in, dx=dh, dw=g_in, db=db, ws=ws)
        d3.rms_norm_backward(dh, self.s, self.gain, self.rstd, ds, dh=ds, dw=dgain, ws=ws)


class Model:
    def __init__(self, vocab=512, width=256, layers=2, tokens=2048, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.table = (torch.randn(vocab, width, generator=gen, device="cuda") * 0.5).to(BF16)
        self.head = (torch.randn(vocab, width, generator=gen, device="cuda") * width ** -0.5).to(BF16)
        self.gain = torch.ones(width, device="cuda")
        self.blocks = [Block(tokens, width, gen) for _ in range(layers)]
        self.dtable, self.dhead, self.dgain = (torch.empty_like(p) for p in (self.table, self.head, self.gain))
        self.grads = [self.dtable, self.dhead, self.dgain] + [g for b in self.blocks for g in b.grads]
        self.x, self.s, self.y, self.ds, self.dh = (new(tokens, width) for _ in range(5))
        self.du, self.logits = new(tokens, 2 * width), new(tokens, vocab)
        self.rstd, self.logp, self.entropy = (new(tokens, dtype=torch.float32) for _ in range(3))
        self.stats, self.norm = new(tokens, 3, dtype=torch.float32), new(1, dtype=torch.float32)
        self.next = new(tokens, 1, dtype=torch.int32)
        self.ws = d3.alloc_workspace(max(
            d3.linear_backward_workspace_size(tokens, width, vocab, dtype=BF16),
            d3.linear_backward_workspace_size(tokens, width, 2 * width, dtype=BF16),
            d3.rms_norm_backward_workspace_size(tokens, width),
            d3.embedding_backward_workspace_size(tokens, vocab, width), d3.grad_norm_workspace_size()))
        self.hp = d3.HParams(f=0.5, mu=0.95, lr=0.02)
        b = self.blocks
        self.groups = [d3.Group([v.w_in for v in b], [v.grads[0] for v in b], [v.m_in for v in b]),
                       d3.Group([v.w_out for v in b], [v.grads[1] for v in b], [v.m_out for v in b])]
        self.step_ws = d3.alloc_workspace(d3.workspace_size(self.groups, self.hp))

    def forward(self, ids, offsets, states=None):
        """The logits of every position; `states`, one tensor a block, are carried on."""
        d3.embedding(ids, self.table, self.x)
        x, stream = self.x, None
        for i, b in enumerate(self.blocks):
            state = None if states is None else states[i]
            x = b.forward(x, stream, offsets, state, state)
            stream = b.s
        d3.rms_norm(x, self.gain, self.y, residual=stream, h=self.s, rstd=self.rstd)
        d3.linear(self.y, self.head, self.logits)
        return self.logits

    def backward(self, ids, targets, offsets, dlogp, dentropy=None):
        """Every gradient, from that of the log probabilities that log_probs left."""
        d3.log_probs_backward(self.logits, targets, self.stats, self.logits, dlogp=dlogp, dentropy=dentropy)
        d3.linear_backward(self.logits, self.y, self.head, dx=self.dh, dw=self.dhead, ws=self.ws)
        d3.rms_norm_backward(self.dh, self.s, self.gain, self.rstd, self.ds, dw=self.dgain, ws=self.ws)
        for b in reversed(self.blocks):
            b.backward(self.ds, offsets, self, self.ws)
        d3.embedding_backward(self.ds, ids, self.dtable, ws=self.ws)

    def train_step(self, ids, targets, offsets, lr=0.2, max_norm=1.0):
        """Mean loss of the batch, on the device."""
        self.forward(ids, offsets)
        d3.log_probs(self.logits, targets, self.logp, stats=self.stats)
        count = (targets >= 0).sum()
        loss = -self.logp.sum() / count
        self.backward(ids, targets, offsets, (-1.0 / count).expand(len(ids)).contiguous())
        d3.clip_grad_norm(self.grads, max_norm, self.norm, ws=self.ws)
        d3.step(self.groups, self.hp, self.step_ws)
        self.table.sub_(self.dtable, alpha=10 * lr)  # the others take plain gradient steps
        self.head.sub_(self.dhead, alpha=lr)
        for p, g in [(self.gain, self.dgain)] + [(b.params[i], b.grads[i]) for b in self.blocks for i in (2, 3)]:
            p.sub_(g, alpha=lr)
        return loss


def generate(model: Model, prompts, length: int):
    """Continues each row of `prompts` by its most probable tokens, one at a time."""
    n, width = len(prompts), model.blocks[0].width
    # The same weights in buffers for n single tokens.
    one = Model(len(model.table), width, len(model.blocks), n)
    for a, b in zip([one.table, one.head, one.gain] + [p for v in one.blocks for p in v.params],
                    [model.table, model.head, model.gain] + [p for v in model.blocks for p in v.params]):
        a.copy_(b)
    states = [torch.zeros(n, width, device="cuda") for _ in one.blocks]
    offsets = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    got = [prompts[:, i].to(torch.int32) for i in range(prompts.shape[1])]
    for i in range(prompts.shape[1] + length - 1):
        logits = one.forward(got[i], offsets, states)
        if i + 1 >= prompts.shape[1]:
            d3.log_probs(logits, top_ids=one.next)
            got.append(one.next[:, 0].clone())
    return torch.stack(got, 1)


def batch(tokens: int, vocab: int, sequences: int, gen: torch.Generator):
    """Packed counting sequences: ids, the tokens that follow them, offsets."""
    cuts = torch.randint(1, tokens, (sequences - 1,), generator=gen, device="cuda").sort()[0].to(torch.int32)
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), tokens)])
    row = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(offsets, row, right=True) - 1
    start, stride = (torch.randint(1, hi, (sequences,), generator=gen, device="cuda") for hi in (vocab, 8))
    ids = (start[seq] + (row - offsets[seq]) * stride[seq]) % vocab
    targets = torch.where(row + 1 < offsets[seq + 1], (ids + stride[seq]) % vocab, PAD)
    return ids, targets, offsets


def train(steps=60, tokens=2048, vocab=512, width=256, layers=2, seed=0):
    """The trained model and the losses of its steps."""
    model = Model(vocab, width, layers, tokens, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = [model.train_step(*batch(tokens, vocab, 16, gen)) for _ in range(steps)]
    d3.device_status()
    return model, [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 60), ("tokens", 2048), ("vocab", 512), ("width", 256), ("layers", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    model, losses = train(**vars(ap.parse_args()))
    for i, loss in enumerate(losses):
        print(f"step {i:3d}  loss {loss:.4f}")
    start = torch.tensor([[5, 7, 9], [100, 101, 102]], device="cuda")
    print(generate(model, start, 6).tolist())
