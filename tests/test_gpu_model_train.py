"""The model operators together with the layer operators and the step, as a training
program and a generating one call them."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def forward64(m, p, ids, offsets):
    """The logits in float64 from the parameters p."""
    table, head, gain, blocks = p
    norm = lambda s, g: s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * g  # noqa: E731
    s = table[ids.clamp(min=0)] * (ids >= 0)[:, None]
    for w_in, w_out, b_in, g in blocks:
        u = norm(s, g) @ w_in.t() + b_in
        width = u.shape[1] // 2
        a = torch.sigmoid(u[:, :width])
        rows, starts, h = [], set(offsets.tolist()), None
        for t in range(len(u)):
            if t in starts:
                h = torch.zeros_like(u[0, :width])
            h = a[t] * h + (1 - a[t]) * u[t, width:]
            rows.append(h)
        s = s + torch.stack(rows) @ w_out.t()
    return norm(s, gain) @ head.t()


def test_gradients_against_autograd(cuda_lib, ex):
    tokens, vocab, width = 120, 90, 64
    m = ex.Model(vocab, width, 2, tokens, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids, targets, offsets = ex.batch(tokens, vocab, 5, gen)
    ids[7] = ex.PAD
    p = [v.double().requires_grad_() for v in (m.table, m.head, m.gain)]
    p.append([[v.double().requires_grad_() for v in b.params] for b in m.blocks])
    logits = forward64(m, p, ids, offsets)
    lp = torch.log_softmax(logits, 1)
    there = targets >= 0
    dlogp, dentropy = torch.randn(tokens, device="cuda"), 0.3 * torch.randn(tokens, device="cuda")
    logp = lp.gather(1, targets.clamp(min=0)[:, None])[:, 0] * there
    entropy = -(lp.exp() * lp).sum(1)
    ((dlogp.double() * logp).sum() + (dentropy.double() * entropy).sum()).backward()

    assert rel(m.forward(ids, offsets), logits.detach()) < 0.02
    d3.log_probs(m.logits, targets, m.logp, entropy=m.entropy, stats=m.stats)
    # Logits of unit size, off by a few roundings of 2^-8 each.
    assert (m.logp - logp).abs().max() < 0.1 and (m.entropy - entropy).abs().max() < 0.1
    m.backward(ids, targets, offsets, dlogp, dentropy)
    # Each value is rounded to bf16 a few times on its way through a block.
    for got, want in zip(m.grads, p[:3] + [v for b in p[3] for v in b]):
        assert rel(got, want.grad) < 0.03


def test_training_and_generating_run(cuda_lib, ex):
    model, losses = ex.train(steps=4, tokens=300, vocab=100, width=64, layers=2)
    assert len(losses) == 4 and all(v == v and v < 20 for v in losses)
    assert float(model.norm) > 0
    prompts = torch.tensor([[1, 2, 3], [9, 7, 5]], device="cuda")
    got = ex.generate(model, prompts, 5)
    assert got.shape == (2, 8) and torch.equal(got[:, :3], prompts.int()) and ((got >= 0) & (got < 100)).all()


def test_token_by_token_is_the_whole_sequence(cuda_lib, ex):
    """The states that generation carries give the logits of one pass over the sequence."""
    n, length, vocab, width = 3, 9, 80, 64
    whole, one = ex.Model(vocab, width, 2, n * length, seed=1), ex.Model(vocab, width, 2, n, seed=1)
    ids = torch.randint(0, vocab, (n, length), device="cuda")
    logits = whole.forward(ids.flatten(), torch.arange(n + 1, dtype=torch.int32, device="cuda") * length).clone()
    states = [torch.zeros(n, width, device="cuda") for _ in one.blocks]
    step = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    for t in range(length):
        got = one.forward(ids[:, t].contiguous(), step, states)
        # The same values rounded at the same places, from states not rounded in between.
        assert rel(got, logits[t::length].double()) < 0.02


def test_a_step_captured_in_a_graph(cuda_lib, ex):
    """A whole training step replayed: the same bits as eager ones."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    batches = [ex.batch(300, 100, 4, gen) for _ in range(3)]
    eager, graph = (ex.Model(100, 64, 2, 300, seed=0) for _ in range(2))
    ids, targets, offsets = (v.clone() for v in batches[0])
    losses = [eager.train_step(*batches[0]), graph.train_step(ids, targets, offsets)]
    assert torch.equal(*losses)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = graph.train_step(ids, targets, offsets)
    for b in batches[1:]:
        for to, v in zip((ids, targets, offsets), b):
            to.copy_(v)
        g.replay()
        want = eager.train_step(*b)
        torch.cuda.synchronize()
        assert torch.equal(loss, want)
        assert all(torch.equal(x, y) for x, y in zip(eager.grads, graph.grads))
        assert torch.equal(eager.blocks[1].w_in, graph.blocks[1].w_in)


def test_first_calls_inside_a_capture(cuda_lib, ex):
    """A process whose very first calls are captured: nothing in them needs an earlier one."""
    code = """
import torch
import matrix_orthogonalizing_optimizer_shape_gb300 as d3
T, D, V = 5000, 64, 300
x = torch.randn(T, D, device="cuda").bfloat16()
ids = torch.randint(0, V, (T,), device="cuda")
h, dz, dx, logits, dl = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.randn(T, V, device="cuda"), torch.empty(T, V, device="cuda")
table, y = torch.empty(V, D, device="cuda"), torch.empty_like(x)
logp, stats, norm = torch.empty(T, device="cuda"), torch.empty(T, 3, device="cuda"), torch.empty(1, device="cuda")
ws = d3.alloc_workspace(max(d3.embedding_backward_workspace_size(T, V, D), d3.grad_norm_workspace_size()))
top = torch.empty(T, 4, device="cuda", dtype=torch.int32)
def go():
    d3.recurrence(x, x, h)
    d3.recurrence_backward(x, x, x, h, dz, dx)
    d3.embedding_backward(x, ids, table, ws=ws)
    d3.embedding(ids, table, y)
    d3.log_probs(logits, ids, logp, stats=stats, top_ids=top)
    d3.log_probs_backward(logits, ids, stats, dl, dlogp=logp)
    d3.clip_grad_norm([dl, y], 1.0, norm, ws=ws)
outs = (h, dz, dx, table, y, logp, stats, top, dl, norm)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    go()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
go()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
d3.device_status()
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
