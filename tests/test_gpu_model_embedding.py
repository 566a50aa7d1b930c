"""Token embedding and its gradient against float64 forms."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import (TINY, TYPES, U, check, dev, embedding_grad_ref, embedding_ref, host, numbers, out, sum_bound,
                        untouched)

pytestmark = pytest.mark.gpu

# tokens, vocab, cols
SHAPES = [(1, 1, 1), (1, 50, 8), (7, 3, 33), (64, 1000, 256), (129, 7, 1000), (300, 300, 2047), (2500, 40, 24),
          (5000, 70000, 8), (40, 300000, 8)]


def draw_ids(rng, tokens, vocab):
    ids = rng.integers(0, vocab, tokens)
    ids[rng.random(tokens) < 0.3] = rng.integers(0, vocab)  # one frequent token
    ids[rng.random(tokens) < 0.1] = rng.choice([-1, vocab, -100, 2 ** 31 - 1])
    return ids


def workspace(tokens, vocab, cols):
    ws = d3.alloc_workspace(d3.embedding_backward_workspace_size(tokens, vocab, cols))
    return ws.fill_(255)  # NaN and -1 wherever a call reads what it did not write


@pytest.mark.parametrize("table_type", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols", SHAPES)
def test_embedding(cuda_lib, table_type, dtype, tokens, vocab, cols):
    rng = np.random.default_rng(tokens + 7 * vocab + 31 * cols)
    ids, values = draw_ids(rng, tokens, vocab), rng.standard_normal((vocab, cols))
    for bits, pad, shift, scale in ((64, 0, 0, 1.0), (32, 3, 1, 1.7), (32, 8, 8, -2.0)):
        table = dev(values, table_type, pad, shift)
        y, buf = out(tokens, cols, dtype, pad, shift)
        d3.embedding(numbers(ids, bits), table, y, scale=scale)
        want = embedding_ref(ids, host(table), float(np.float32(scale)))
        check(host(y), want, np.abs(want) * (2.0 ** -24 + 1.001 * U[dtype]) + TINY[dtype], "y")
        assert untouched(y, buf)


@pytest.mark.parametrize("table_type", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols", SHAPES)
def test_embedding_backward(cuda_lib, table_type, dtype, tokens, vocab, cols):
    rng = np.random.default_rng(tokens + 7 * vocab + 31 * cols)
    ids, grad = draw_ids(rng, tokens, vocab), rng.standard_normal((tokens, cols))
    for bits, pad, shift, scale, accumulate in ((64, 0, 0, 1.0, False), (32, 3, 1, 1.7, True), (32, 8, 8, 1.0, True),
                                                (64, 1, 0, -0.5, False)):
        dy = dev(grad, dtype, pad, shift)
        dtable, buf = out(vocab, cols, table_type, pad, shift)
        d3.embedding_backward(dy, numbers(ids, bits), dtable, scale=scale, accumulate=accumulate,
                              ws=workspace(tokens, vocab, cols))
        want, mag, n = embedding_grad_ref(host(dy), ids, vocab, float(np.float32(scale)))
        if accumulate:
            want = want + 7.0
        tol = sum_bound(1) * (n[:, None] + 2) * mag + (2.0 ** -23 + 1.001 * U[table_type]) * np.abs(want)
        check(host(dtable), want, np.where(n[:, None] > 0, tol + TINY[table_type], 0.0), "dtable")
        assert untouched(dtable, buf)


@pytest.mark.parametrize("tokens,cols,frequent", [(5000, 40, 1.0), (20000, 8, 0.97), (9000, 1001, 0.5), (70000, 8, 1.0)])
def test_runs_over_many_windows(cuda_lib, tokens, cols, frequent):
    """A token that makes up much or all of the batch, between rare ones."""
    rng = np.random.default_rng(tokens)
    ids = np.where(rng.random(tokens) < frequent, 300, rng.integers(0, 1000, tokens))
    # Whole numbers, whose sums are exact in 32 bits in any order.
    dy = dev(rng.integers(-8, 9, (tokens, cols)), "bf16")
    dtable, _ = out(1000, cols, "f32")
    ws = workspace(tokens, 1000, cols)
    d3.embedding_backward(dy, numbers(ids), dtable, ws=ws)
    want, _, _ = embedding_grad_ref(host(dy), ids, 1000, 1.0)
    assert np.array_equal(host(dtable), want)


def test_every_window_boundary(cuda_lib):
    """Runs that end at, before and behind each window's last position."""
    for run in (1, 7, 8, 9, 16, 17, 24, 31):
        ids = np.repeat(np.arange(40), run) * 256  # one group, so that the runs follow one another
        dy = dev(np.arange(len(ids) * 8).reshape(-1, 8) % 251 - 125, "f32")
        dtable, _ = out(40 * 256, 8, "f32")
        d3.embedding_backward(dy, numbers(ids), dtable, ws=workspace(len(ids), 40 * 256, 8))
        want, _, _ = embedding_grad_ref(host(dy), ids, 40 * 256, 1.0)
        assert np.array_equal(host(dtable), want), run


def test_no_tokens_and_only_padding(cuda_lib):
    for tokens in (0, 5):
        dy, ids = torch.ones(tokens, 8, device="cuda"), torch.full((tokens,), -1, device="cuda")
        d3.embedding(ids, torch.ones(4, 8, device="cuda"), dy)
        assert not dy.any()
        for accumulate in (False, True):
            dtable, buf = out(4, 8, "bf16", 3)
            d3.embedding_backward(dy, ids, dtable, accumulate=accumulate, ws=workspace(tokens, 4, 8))
            assert (dtable == (7.0 if accumulate else 0.0)).all() and untouched(dtable, buf)


def test_empty_table(cuda_lib):
    y = torch.ones(3, 8, device="cuda")
    ids, table = torch.tensor([0, 1, -1], device="cuda"), torch.empty(0, 8, device="cuda")
    d3.embedding(ids, table, y)
    assert not y.any()
    d3.embedding_backward(y, ids, table, ws=workspace(3, 0, 8))


def test_nan_and_infinity_stay_with_their_token(cuda_lib):
    ids = numbers([1, 2, 2, 3, 5, -1])
    dy = torch.ones(6, 64, device="cuda", dtype=torch.bfloat16)
    dy[1, 3], dy[3, 4], dy[5] = float("nan"), float("inf"), float("nan")
    dtable, _ = out(6, 64, "bf16")
    d3.embedding_backward(dy, ids, dtable, ws=workspace(6, 6, 64))
    want = torch.zeros(6, 64)
    want[1], want[2], want[3], want[5] = 1, 2, 1, 1
    want[2, 3], want[3, 4] = float("nan"), float("inf")
    assert torch.equal(torch.nan_to_num(dtable.float().cpu(), 9.0), torch.nan_to_num(want, 9.0))
    y, _ = out(6, 64, "bf16")
    d3.embedding(ids, dtable, y)
    assert torch.isnan(y[1, 3]) and torch.isfinite(y[0]).all() and not y[5].any()


def test_offsets_past_32_bits(cuda_lib):
    vocab, cols, tokens = 1100000, 2048, 60
    table = torch.empty(vocab, cols, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(5)
    ids = numbers(np.concatenate([rng.integers(vocab - 40, vocab, tokens - 2), [0, vocab // 2]]))
    table[ids] = torch.randn(tokens, cols, device="cuda").to(table.dtype)
    y = torch.empty(tokens, cols, dtype=torch.bfloat16, device="cuda")
    d3.embedding(ids, table, y)
    assert torch.equal(y, table[ids])
    ws = workspace(tokens, vocab, cols)
    table.fill_(float("nan"))
    d3.embedding_backward(y, ids, table, ws=ws)
    want, mag, n = embedding_grad_ref(host(y), ids.cpu().numpy() - (vocab - 40), 40, 1.0)
    check(host(table[-40:]), want, sum_bound(60) * mag + 1.001 * U["bf16"] * np.abs(want), "dtable")
    assert torch.equal(table[vocab // 2], y[-1]) and not table[1:vocab // 2].any()
    del table
    wide = torch.zeros(5, 1 << 30, dtype=torch.bfloat16, device="cuda")[:, :24]  # rows 2^30 elements apart
    wide.copy_(torch.randn(5, 24, device="cuda"))
    small, _ = out(4, 24, "f32")
    d3.embedding_backward(wide, numbers([3, 1, 3, 3, 0]), small, ws=workspace(5, 4, 24))
    w = wide.float()
    assert torch.equal(small, torch.stack([w[4], w[1], torch.zeros_like(w[0]), w[0] + w[2] + w[3]]))


def test_equal_bits_on_other_streams_and_in_a_graph(cuda_lib):
    tokens, vocab, cols = 6000, 900, 1024
    rng = np.random.default_rng(1)
    ids, dy = numbers(draw_ids(rng, tokens, vocab)), dev(rng.standard_normal((tokens, cols)), "bf16")
    ws = workspace(tokens, vocab, cols)
    first, _ = out(vocab, cols, "f32")
    d3.embedding_backward(dy, ids, first, ws=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again, _ = out(vocab, cols, "f32")
        d3.embedding_backward(dy, ids, again, ws=ws.fill_(255))
    s.synchronize()
    assert torch.equal(first, again)
    y, x = torch.empty_like(dy), torch.empty_like(dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d3.embedding_backward(dy, ids, again, ws=ws)
        d3.embedding(ids, again, y)
    other = numbers(draw_ids(rng, tokens, vocab))
    for v in (ids.clone(), other):  # new ids in the captured call's place
        ids.copy_(v)
        g.replay()
        d3.embedding_backward(dy, v, first, ws=workspace(tokens, vocab, cols))
        d3.embedding(v, first, x)
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(x, y)


def test_frequent_tokens_give_equal_bits_whoever_joins_them(cuda_lib):
    """Runs over many windows are added by whichever block is last: in the same order."""
    rng = np.random.default_rng(2)
    tokens, vocab, cols = 16000, 200, 2048
    ids = numbers(np.minimum((vocab * rng.random(tokens) ** 3).astype(int), vocab - 1))
    dy = dev(rng.standard_normal((tokens, cols)), "bf16")
    ws, first = workspace(tokens, vocab, cols), None
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(out(vocab, cols, "f32")[0], workspace(tokens, vocab, cols)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, (dtable, own) in zip(streams, outs):  # side by side, a workspace each
            with torch.cuda.stream(s):
                d3.embedding_backward(dy, ids, dtable, ws=own)
        torch.cuda.synchronize()
        dtable, _ = out(vocab, cols, "f32")
        d3.embedding_backward(dy, ids, dtable, ws=ws)
        first = dtable if first is None else first
        assert torch.equal(first, dtable) and all(torch.equal(first, d) for d, _ in outs)
