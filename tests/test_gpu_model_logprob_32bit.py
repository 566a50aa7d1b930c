"""Statistics of log probabilities are kept in 32 bits: errors over many rows, beside the
worst case of one that test_gpu_model_logprob.py allows.

Errors of log S, with u = 2^-23, from one row to the next (independent roundings add as
their squares): a thread's sum of n = vocab / 256 + 8 terms, sqrt(n) u / 2 (1.4e-6 at 131072
columns); eleven joins and some ten larger maxima on the way, each an exponential of the
difference of two maxima, at most 10 here: sqrt(21) (2 + 1.5 x 10) u / 2 = 4.7e-6.  Alike in
all rows: the exponential's 2 u and what scale log2 e is off by, 1.5 u / 2 times W = sum p
|s d| (at most 16 here): 1.7e-6; the logarithm's own u / 2 of at most 12: 0.7e-6.  Together
less than 1e-5.  Q / S = -W / s has the same relative errors, and the entropy is log S + s Q
/ S; the target's s d is rounded thrice.  So 1e-5 (1 + |value|) as the root of the mean
square, and four times that for the worst of some hundred rows.

The gradient's elements: p by log p, off by as much and by 1.5 u / 2 |log p|, and the
exponential's 2 u; the entropy's factor log p + H is off by 1e-5 (1 + H + |log p|).
"""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import U, dev, host, log_probs_grad_ref, log_probs_ref, numbers

pytestmark = pytest.mark.gpu

RMS = 1e-5


def rows_of(rng, rows, vocab, size):
    v = size * rng.standard_normal((rows, vocab))
    if size > 1:
        v[np.arange(rows), rng.integers(0, vocab, rows)] += 8
    return v


def rms(got, want):
    return float(np.sqrt(np.mean(((got - want) / (1 + np.abs(want))) ** 2)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,size,scale", [
    (100, 131072, 2.0, 1.0), (100, 131072, 0.01, 1.0), (300, 32001, 2.0, 1.25), (300, 32001, 0.01, 1.25),
    (1200, 5003, 3.0, 0.7), (1200, 5003, 0.01, 1.0)])
def test_statistics_over_many_rows(cuda_lib, dtype, rows, vocab, size, scale):
    rng = np.random.default_rng(vocab)
    logits, targets = dev(rows_of(rng, rows, vocab, size), dtype), rng.integers(0, vocab, rows)
    new = lambda *n: torch.empty(*n, device="cuda")  # noqa: E731
    logp, entropy, stats, top = new(rows), new(rows), new(rows, 3), new(rows, 20)
    d3.log_probs(logits, numbers(targets), logp, scale=scale, entropy=entropy, stats=stats, top_values=top)
    want, ent, lp = log_probs_ref(host(logits), targets, float(np.float32(scale)))
    assert -lp.max(1).min() < 12 and (np.exp(lp) * np.abs(lp - lp.max(1, keepdims=True))).sum(1).max() < 16
    best = -np.partition(-lp, 19, 1)[:, :20]
    for got, right in ((host(logp), want), (host(entropy), ent), (host(stats)[:, 1], -lp.max(1)),
                       (host(top), -np.sort(-best, 1))):
        off = np.abs(got - right) / (1 + np.abs(right))
        assert rms(got, right) <= RMS and off.max() <= 4 * RMS, (rms(got, right), off.max())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,size,scale", [(40, 131072, 2.0, 1.0), (150, 32001, 2.0, 1.25), (150, 32001, 0.01, 1.25)])
def test_gradient_over_many_rows(cuda_lib, dtype, rows, vocab, size, scale):
    rng = np.random.default_rng(vocab + 1)
    logits, targets = dev(rows_of(rng, rows, vocab, size), dtype), rng.integers(0, vocab, rows)
    stats, d = torch.empty(rows, 3, device="cuda"), torch.empty_like(logits)
    g, e = (torch.from_numpy(256 * rng.standard_normal(rows)).float().cuda() for _ in range(2))
    s32 = float(np.float32(scale))
    d3.log_probs(logits, numbers(targets), scale=scale, stats=stats)
    _, h, lp = log_probs_ref(host(logits), targets, s32)
    p = np.exp(lp)
    for dentropy in (None, e):
        d3.log_probs_backward(logits, numbers(targets), stats, d, dlogp=g, dentropy=dentropy, scale=scale)
        want = log_probs_grad_ref(host(logits), targets, s32, host(g), None if dentropy is None else host(e))
        # What p and, of the entropy's term, p (log p + H) may be off by, element by element.
        part = np.abs(host(g))[:, None] * p
        if dentropy is not None:
            part = part + 2 * np.abs(host(e))[:, None] * p * (1 + h[:, None] + np.abs(lp))
        off = RMS * (1 + 0.01 * np.abs(lp)) * part * s32 + 1.001 * U[dtype] * np.abs(want) + {"f16": 2.0 ** -25}.get(dtype, 0.0)
        got = host(d)
        live = (np.arange(vocab) != targets[:, None])  # the target's own element is rounded against g
        rows_off = np.sqrt((((got - want) * live) ** 2).sum(1)) / np.sqrt((off ** 2).sum(1))
        assert rows_off.max() <= 4 and np.sqrt(np.mean(rows_off ** 2)) <= 1, rows_off
        at = np.arange(rows), targets
        assert (np.abs(got - want)[at] <= 4 * off[at] + 2.0 ** -22 * s32 * np.abs(host(g))).all()
