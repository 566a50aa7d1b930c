"""States of the recurrence that are not finite: every later one of the channel and the
sequence is not finite either (infinity or NaN), and no other sequence or channel sees it,
wherever the row falls among the rows of threads, lanes and blocks.  (a h + b of an
infinite h is infinite for 0 < a and NaN for a = 0, and so are the composed forms: -D inf
+ inf and 0 inf are NaN, A inf is infinite.  All tests are exact.)"""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import host, numbers

pytestmark = pytest.mark.gpu

INF = float("inf")
# Rows a thread of one and of several, boxes, cells and registers, clusters of several blocks.
SHAPES = [("bf16", 300, 64), ("f32", 2600, 130), ("bf16", 9000, 72), ("f16", 700, 33), ("bf16", 40, 4096), ("f32", 5000, 64)]
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def places(tokens):
    """Rows about the borders of threads' rows, and of blocks' ones."""
    return sorted({p for p in (0, 1, 3, 7, 8, 9, 15, 16, 17, 31, 100, 127, 128, 255, 256, 511, tokens // 2, tokens - 2,
                               tokens - 1) if p < tokens})


@pytest.mark.parametrize("gate", [-90.0, -2.0, 0.0, 3.0, 20.0, INF, -INF])
@pytest.mark.parametrize("dtype,tokens,channels", SHAPES)
def test_no_state_after_an_infinite_one_is_finite(cuda_lib, dtype, tokens, channels, gate):
    """Channel i meets infinity in x at the i-th place, and a state before the second
    sequence is infinite; `gate` is what the rows behind them have."""
    e, cut = TORCH[dtype], tokens // 3
    off = numbers([0, cut, tokens], 32)
    spots = places(tokens)[:channels - 1]
    z = torch.full((tokens, channels), gate, dtype=e, device="cuda")
    x = torch.randn(tokens, channels, device="cuda").to(e)
    first = torch.randn(2, channels, device="cuda")
    first[1, channels - 1] = -INF
    for i, at in enumerate(spots):
        x[at, i], z[at, i] = INF, 0.0
    h, last = torch.empty_like(x), torch.empty_like(first)
    d3.recurrence(z, x, h, offsets=off, first=first, last=last)
    finite = np.isfinite(host(h))
    want = np.ones((tokens, channels), dtype=bool)
    for i, at in enumerate(spots):
        want[at:cut if at < cut else tokens, i] = False
        assert h[at, i] == INF
    want[cut:, channels - 1] = False
    assert np.array_equal(finite, want)
    assert np.array_equal(np.isfinite(host(last)), want[[cut - 1, tokens - 1]])


@pytest.mark.parametrize("gate", [-90.0, -2.0, 0.0, 3.0, 20.0, INF, -INF])
@pytest.mark.parametrize("dtype,tokens,channels", SHAPES)
def test_no_gradient_before_an_infinite_one_is_finite(cuda_lib, dtype, tokens, channels, gate):
    e, cut = TORCH[dtype], tokens // 3
    off = numbers([0, cut, tokens], 32)
    spots = [tokens - 1 - p for p in places(tokens)][:channels - 1]
    z = torch.full((tokens, channels), gate, dtype=e, device="cuda")
    x, h, dh = (torch.randn(tokens, channels, device="cuda").to(e) for _ in range(3))
    dlast = torch.randn(2, channels, device="cuda")
    dlast[0, channels - 1] = INF
    for i, at in enumerate(spots):
        dh[at, i], z[at, i] = -INF, 0.0
    dz, dx, dfirst = torch.empty_like(x), torch.empty_like(x), torch.empty_like(dlast)
    d3.recurrence_backward(dh, z, x, h, dz, dx, offsets=off, dlast=dlast, dfirst=dfirst)
    want = np.ones((tokens, channels), dtype=bool)
    for i, at in enumerate(spots):
        want[0 if at < cut else cut:at + 1, i] = False
        assert dx[at, i] == -INF
    want[:cut, channels - 1] = False
    assert np.array_equal(np.isfinite(host(dx)), want)
    assert np.array_equal(np.isfinite(host(dz)), want)
    assert np.array_equal(np.isfinite(host(dfirst)), want[[0, cut]])
