"""Log probabilities, entropy, alternatives and their gradient against float64 forms.

Bounds, with u = 2^-23.  An exponential e^(s d) of a difference d is off by (2 + 2 |s d|) u
relative: the instruction by 2 u, its argument by three roundings.  Terms with
s d < -30 are below 2^-43 of the sum, so the sum S of positive terms is off by at
most (2 + 60 + additions) u, where a thread adds at most vocab / 256 + 8 terms and
joins take 16 more roundings each with an exponential: ADDS below.  log S is off
by as much and a rounding of itself; the largest |s d| (the target's) adds its own.
Q / S = sum p d has terms of at most |s d| p, each off by the same relative amount.
"""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import (TINY, TYPES, U, check, dev, host, log_probs_grad_ref, log_probs_ref, numbers, out, top_ref,
                        untouched)

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 131072), (3, 7), (2, 33), (5, 1000), (70, 32001), (1300, 257), (4, 5003), (33, 8192)]


def adds(vocab):
    return (62 + vocab / 256 + 8 + 16 * 64) * 2.0 ** -23


def make(rng, rows, vocab, dtype, pad=0, shift=0, masked=False, size=3.0):
    v = size * rng.standard_normal((rows, vocab))
    if masked:
        v[rng.random((rows, vocab)) < 0.3] = -np.inf
        v[rng.random((rows, vocab)) < 0.1] = float(torch.finfo(torch.float16).min)
    targets = rng.integers(0, vocab, rows)
    targets[rng.random(rows) < 0.2] = -100
    return dev(v, dtype, pad, shift), targets


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_log_probs(cuda_lib, dtype, rows, vocab):
    rng = np.random.default_rng(rows * 7 + vocab)
    for pad, shift, masked, scale, bits, k in ((0, 0, False, 1.0, 64, 0), (3, 1, True, 1.25, 32, 20), (8, 0, False, 0.1, 32, 1),
                                               (1, 5, True, 2.0, 64, 32)):
        k = min(k, vocab)
        logits, targets = make(rng, rows, vocab, dtype, pad, shift, masked)
        new = lambda *n: torch.full(n, 9.0, device="cuda")  # noqa: E731
        logp, entropy, stats = new(rows), new(rows), new(rows, 3)
        tv, ti = (new(rows, k), torch.full((rows, k), -7, dtype=torch.int32, device="cuda")) if k else (None, None)
        d3.log_probs(logits, numbers(targets, bits), logp, scale=scale, entropy=entropy, stats=stats, top_values=tv,
                     top_ids=ti)
        s32 = float(np.float32(scale))
        want, ent, lp = log_probs_ref(host(logits), targets, s32)
        size = np.where(np.isfinite(want), np.abs(want), 0.0)
        check(np.nan_to_num(host(logp), neginf=-1e30), np.nan_to_num(want, neginf=-1e30), adds(vocab) + 4 * size * 2.0 ** -23, "logp")
        check(host(entropy), ent, 4 * adds(vocab) * (1 + ent), "entropy")
        top = host(logits).max(1)
        live = ~np.isneginf(top)
        assert (host(stats)[live, 0] == top[live]).all() and np.array_equal(host(stats)[:, 2], host(entropy))
        with np.errstate(invalid="ignore"):
            check(host(stats)[live, 1], -lp.max(1)[live], adds(vocab) * 2, "log sum")
        if k:
            ids = top_ref(host(logits), k)
            assert np.array_equal(ti.cpu().numpy(), ids)
            wv = np.take_along_axis(lp, ids, 1)
            ok = np.isfinite(wv)
            assert np.array_equal(np.isneginf(host(tv)), ~ok)
            check(host(tv)[ok], wv[ok], (adds(vocab) + 4 * np.abs(wv) * 2.0 ** -23)[ok], "top values")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_log_probs_backward(cuda_lib, dtype, rows, vocab):
    rng = np.random.default_rng(rows * 7 + vocab)
    for pad, shift, masked, scale, bits, ent in ((0, 0, False, 1.0, 64, False), (3, 1, True, 1.25, 32, True), (8, 0, True, 1.0, 64, True)):
        logits, targets = make(rng, rows, vocab, dtype, pad, shift, masked)
        t = numbers(targets, bits)
        stats = torch.empty(rows, 3, device="cuda")
        d3.log_probs(logits, t, torch.empty(rows, device="cuda"), scale=scale, stats=stats)
        dlogp = torch.from_numpy(rng.standard_normal(rows)).float().cuda()
        dent = torch.from_numpy(rng.standard_normal(rows)).float().cuda() if ent else None
        s32 = float(np.float32(scale))
        want = log_probs_grad_ref(host(logits), targets, s32, host(dlogp), host(dent) if ent else None)
        # p is off by adds + 2 units and its exponent's; each term as p, the entropy's factor by adds more.
        _, h, lp = log_probs_ref(host(logits), targets, s32)
        p = np.exp(lp)
        far = np.where(p > 0, np.abs(np.where(p > 0, lp, 0.0)), 0.0)
        rel = 2 * adds(vocab) + 6 * far * 2.0 ** -23
        part = np.abs(host(dlogp))[:, None] * (p + (np.arange(vocab) == targets[:, None]) * 1.0) * s32
        if ent:
            part = part + 4 * np.abs(host(dent))[:, None] * p * (far + h[:, None] + 1) * s32
        tol = rel * part + 1.001 * U[dtype] * np.abs(want) + TINY[dtype] + 2.0 ** -120
        for place in (False, True):
            d, buf = out(rows, vocab, dtype, pad, shift + (0 if pad else 8))
            if place:
                d, buf = logits, None
            d3.log_probs_backward(logits, t, stats, d, dlogp=dlogp, dentropy=dent, scale=scale)
            check(host(d), want, tol, "dlogits")
            assert place or untouched(d, buf)


def test_rows_at_other_places_of_a_piece(cuda_lib):
    """Input and output rows that begin at different offsets from 16 bytes."""
    rng = np.random.default_rng(4)
    for shift in range(8):
        logits, targets = make(rng, 6, 3001, "bf16", 5, shift)
        stats, dlogp = torch.empty(6, 3, device="cuda"), torch.ones(6, device="cuda")
        d3.log_probs(logits, numbers(targets), torch.empty(6, device="cuda"), stats=stats)
        a, abuf = out(6, 3001, "bf16", 2, 3)
        b, _ = out(6, 3001, "bf16", 5, shift)
        d3.log_probs_backward(logits, numbers(targets), stats, a, dlogp=dlogp)
        d3.log_probs_backward(logits, numbers(targets), stats, b, dlogp=dlogp)
        assert torch.equal(a, b) and untouched(a, abuf)


@pytest.mark.parametrize("vocab", [40, 5003, 131072])
def test_special_rows(cuda_lib, vocab):
    """Everything masked, by infinity and by the type's lowest value; one token left; equal
    logits; far apart; NaN and infinity."""
    inf, nan, low = float("inf"), float("nan"), float(torch.finfo(torch.bfloat16).min)
    x = torch.randn(10, vocab, device="cuda").to(torch.bfloat16)
    x[0], x[1], x[2] = -inf, low, -inf
    x[2, 17] = -3.0
    x[3] = 2.5
    x[4, :] = -low
    x[4, 1::2] = low
    x[5, 9], x[6, 9], x[7] = nan, inf, nan
    x[8] = torch.where(torch.arange(vocab, device="cuda") < 5, x[8], -inf)
    x[9, 3] = -inf
    targets = torch.tensor([1, 2, 17, 5, 0, 1, 9, 0, 30, 3], device="cuda")
    logp, entropy, stats = (torch.empty(10, n, device="cuda").squeeze(1) for n in (1, 1, 3))
    tv, ti = torch.empty(10, 12, device="cuda"), torch.empty(10, 12, dtype=torch.int32, device="cuda")
    d3.log_probs(x, targets, logp, entropy=entropy, stats=stats, top_values=tv, top_ids=ti)
    want, ent, lp = log_probs_ref(host(x), targets.cpu().numpy(), 1.0)
    fine = [i for i in range(10) if i not in (5, 6, 7)]
    assert np.array_equal(np.isneginf(host(logp))[fine], np.isneginf(want)[fine]) and logp[0] == -inf and logp[8] == -inf
    ok = [i for i in fine if np.isfinite(want[i])]
    check(host(logp)[ok], want[ok], adds(vocab) * (1 + np.abs(want[ok])), "logp")
    check(host(entropy)[fine], ent[fine], 4 * adds(vocab) * (1 + ent[fine]), "entropy")
    assert entropy[0] == 0 and entropy[2] == 0 and logp[2] == 0
    assert torch.isnan(logp[[5, 6, 7]]).all() and torch.isnan(entropy[[5, 6, 7]]).all() and torch.isnan(tv[[5, 6, 7]]).all()
    assert np.array_equal(ti.cpu().numpy(), top_ref(host(x), 12))
    assert (tv[0] == -inf).all() and (tv[8, 5:] == -inf).all() and torch.isfinite(tv[8, :5]).all()
    d = torch.full_like(x, 7.0)
    g, e = torch.ones(10, device="cuda"), torch.full((10,), 0.5, device="cuda")
    targets[7] = -1
    e[7] = 0
    d3.log_probs_backward(x, targets, stats, d, dlogp=g, dentropy=e)
    assert not d[0].any() and not d[7].any() and torch.isnan(d[5:7]).all() and not d[2].any()
    wd = log_probs_grad_ref(host(x)[fine], targets.cpu().numpy()[fine], 1.0, np.ones(7), np.full(7, 0.5))
    check(host(d)[fine], wd, 8 * adds(vocab) * (np.abs(wd) + 2.0 / vocab) + 1.001 * U["bf16"] * np.abs(wd) + 2.0 ** -120, "dlogits")


@pytest.mark.parametrize("rows,vocab", [(3, 131072), (2, 5003), (1300, 40007)])
@pytest.mark.parametrize("dtype", TYPES)
def test_alternatives_among_equal_logits(cuda_lib, dtype, rows, vocab):
    """Few values, so that equal logits reach far along a row: masked ones, the type's lowest, one value, NaN."""
    rng = np.random.default_rng(vocab)
    low = float(torch.finfo(torch.float16).min)
    for values, p in (([-np.inf, 1.0, 2.0], [0.9999, 0.00005, 0.00005]), ([-np.inf, low, 3.0], [0.5, 0.4999, 0.0001]),
                      ([0.0, -0.0, 1.0], [0.5, 0.4999, 0.0001]), ([5.0, 4.0, 3.0], [0.001, 0.01, 0.989]),
                      ([-np.inf, np.nan, 1.0], [0.01, 0.989, 0.001]), ([np.nan, np.nan, -np.inf], [0.5, 0.4999, 0.0001])):
        logits = dev(rng.choice(values, size=(min(rows, 40), vocab), p=p), dtype, 3, 1)
        if rows > 40:
            logits = logits.repeat(rows // 40 + 1, 1)[:rows]
        for k in (1, 20, 32):
            ids = torch.empty(rows, k, dtype=torch.int32, device="cuda")
            d3.log_probs(logits, top_ids=ids)
            want = top_ref(host(logits[:40]), k)
            got = ids.cpu().numpy()
            assert np.array_equal(got[:len(want)], want) and np.array_equal(got, want[np.arange(rows) % len(want)])


def test_each_result_alone(cuda_lib):
    """A result does not depend on which others are asked for, and each may be left out."""
    rng = np.random.default_rng(0)
    for rows, vocab in ((2, 50001), (2000, 500)):
        logits, targets = make(rng, rows, vocab, "bf16")
        t = numbers(targets)
        f = lambda *n: torch.empty(*n, device="cuda")  # noqa: E731
        logp, entropy, stats, tv, ti = f(rows), f(rows), f(rows, 3), f(rows, 7), f(rows, 7).int()
        d3.log_probs(logits, t, logp, entropy=entropy, stats=stats, top_values=tv, top_ids=ti)
        logp2, entropy2, stats2, tv2, ti2 = f(rows), f(rows), f(rows, 3), f(rows, 7), f(rows, 7).int()
        d3.log_probs(logits, t, logp2)
        d3.log_probs(logits, entropy=entropy2)
        d3.log_probs(logits, stats=stats2)
        d3.log_probs(logits, top_values=tv2)
        d3.log_probs(logits, top_ids=ti2)
        d3.log_probs(logits)
        for a, b in ((logp, logp2), (entropy, entropy2), (stats, stats2), (tv, tv2), (ti, ti2)):
            assert torch.equal(a, b)
        d, d2 = torch.empty_like(logits), torch.empty_like(logits)
        g = torch.randn(rows, device="cuda")
        d3.log_probs_backward(logits, None, stats, d, dentropy=g)
        d3.log_probs_backward(logits, numbers(np.full(rows, -1)), stats, d2, dlogp=g, dentropy=g)
        assert torch.equal(d, d2)
        d3.log_probs_backward(logits, None, stats, d)
        assert not d.any()


def test_large_logits_keep_their_differences(cuda_lib):
    """An offset common to a row's logits changes nothing."""
    x = torch.randn(40, 3000, device="cuda").mul(64).round().div(64)
    t = torch.randint(0, 3000, (40,), device="cuda")
    a, b, ea, eb = (torch.empty(40, device="cuda") for _ in range(4))
    d3.log_probs(x, t, a, entropy=ea, scale=0.7)
    d3.log_probs(x + 16384, t, b, entropy=eb, scale=0.7)
    assert torch.equal(a, b) and torch.equal(ea, eb)


def test_gradient_against_differences(cuda_lib):
    rng = np.random.default_rng(6)
    rows, vocab, scale = 20, 700, 1.5
    x, targets = 2 * rng.standard_normal((rows, vocab)), rng.integers(0, vocab, rows)
    x[3, 5], targets[4] = -np.inf, -100
    g, e = rng.standard_normal(rows), rng.standard_normal(rows)

    def value(v):
        logp, entropy, _ = log_probs_ref(v, targets, scale)
        return float((g * logp).sum() + (e * entropy).sum())

    t = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    stats, d = torch.empty(rows, 3, device="cuda"), torch.empty(rows, vocab, device="cuda")
    targets[targets == 5] = 6
    d3.log_probs(t(x), numbers(targets), scale=scale, stats=stats)
    d3.log_probs_backward(t(x), numbers(targets), stats, d, dlogp=t(g), dentropy=t(e), scale=scale)
    v = rng.standard_normal(x.shape)
    num = (value(x + 1e-5 * v) - value(x - 1e-5 * v)) / 2e-5
    terms = host(d) * v
    assert abs(terms.sum() - num) < 2e-6 * np.abs(terms).sum() and (host(d)[3, 5] == 0)


def test_offsets_past_32_bits(cuda_lib):
    big = torch.zeros(3, 1 << 31, dtype=torch.bfloat16, device="cuda")
    x = big[:, :5000]
    x.copy_(torch.randn(3, 5000, device="cuda"))
    t = numbers([1, 4999, 7])
    a, b, stats = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, 3, device="cuda")
    ids, ids2 = (torch.empty(3, 9, dtype=torch.int32, device="cuda") for _ in range(2))
    d3.log_probs(x, t, a, stats=stats, top_ids=ids)
    d3.log_probs(x.contiguous(), t, b, top_ids=ids2)
    assert torch.equal(a, b) and torch.equal(ids, ids2)
    d = torch.empty(3, 5000, dtype=torch.bfloat16, device="cuda")
    d3.log_probs_backward(x.contiguous(), t, stats, d, dlogp=a)
    d3.log_probs_backward(x, t, stats, x, dlogp=a)
    assert torch.equal(d, x)


def test_no_rows(cuda_lib):
    e = torch.empty(0, 9, device="cuda")
    t, v = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    d3.log_probs(e, t, v, top_values=torch.empty(0, 3, device="cuda"))
    d3.log_probs_backward(e, t, torch.empty(0, 3, device="cuda"), e, dlogp=v)


def test_equal_bits_on_other_streams_and_in_a_graph(cuda_lib):
    rng = np.random.default_rng(9)
    for rows, vocab in ((1, 131072), (700, 3001)):
        logits, targets = make(rng, rows, vocab, "bf16")
        t = numbers(targets)
        f = lambda *n: torch.empty(*n, device="cuda")  # noqa: E731
        dlogp = torch.randn(rows, device="cuda")

        def go(o):
            d3.log_probs(logits, t, o[0], entropy=o[1], stats=o[2], top_values=o[3], top_ids=o[4])
            d3.log_probs_backward(logits, t, o[2], o[5], dlogp=dlogp)

        one, two = ([f(rows), f(rows), f(rows, 3), f(rows, 20), f(rows, 20).int(), torch.empty_like(logits)] for _ in range(2))
        go(one)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            go(two)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(two)
        logits.copy_(torch.randn(rows, vocab, device="cuda"))
        g.replay()
        go(one)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(one, two))
