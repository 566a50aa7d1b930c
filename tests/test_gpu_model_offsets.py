"""Offsets that do not ascend give undefined values in the rows of the recurrence, but both
passes end and write nothing outside their matrices and states: every result lies in a
buffer whose other elements are marked.  (All reads are of sequences from 0 to n - 1 and
rows that the kernels limit to the matrices'.)"""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import dev, numbers, out, untouched

pytestmark = pytest.mark.gpu

LISTS = {
    "back": [0, 500, 100, 400], "outside": [-5, 900, -7, 2000], "reversed": [400, 0], "one place": [300] * 4,
    "extremes": [2 ** 31 - 1, -2 ** 31, 5], "behind the rows": [400, 500, 600], "negative": [-9, -5, -1, 0],
    "many shuffled": None, "many outside": None,  # read from global memory
}


def offsets_of(name, tokens):
    if LISTS[name] is not None:
        return LISTS[name]
    rng = np.random.default_rng(len(name))
    return list(rng.permutation(1500) % (tokens + 1) if name == "many shuffled" else rng.integers(-2 ** 31, 2 ** 31, 1300))


def states(n, channels):
    """A [n, channels] state inside a marked buffer, and the buffer."""
    buf = torch.full((n + 2, channels), 7.0, device="cuda")
    return buf[1:-1], buf


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("dtype,tokens,channels,pad,shift", [("bf16", 400, 66, 2, 0), ("f32", 400, 33, 0, 3),
                                                       ("bf16", 20, 4096, 0, 0), ("f16", 5000, 128, 8, 0),
                                                       ("bf16", 6000, 64, 0, 8)])
def test_nothing_outside_is_written(cuda_lib, name, dtype, tokens, channels, pad, shift):
    off = numbers(offsets_of(name, tokens), 32)
    n = len(off) - 1
    ones = lambda: dev(np.ones((tokens, channels)), dtype, pad)  # noqa: E731
    z, x = ones(), ones()
    (h, hb), (dz, zb), (dx, xb) = (out(tokens, channels, dtype, pad, shift) for _ in range(3))
    for given in (True, False):
        (first, fb), (last, lb), (dlast, eb), (dfirst, db) = (states(n, channels) for _ in range(4))
        d3.recurrence(z, x, h, offsets=off, first=first if given else None, last=last)
        d3.recurrence_backward(x, z, x, x, dz, dx, offsets=off, first=first if given else None,
                               dlast=dlast if given else None, dfirst=dfirst)
        for v, buf in ((h, hb), (dz, zb), (dx, xb)):
            assert untouched(v, buf)
        for buf in (fb, lb, eb, db):
            assert (buf[[0, -1]] == 7).all()
        assert (first == 7).all() and (dlast == 7).all()
        d3.recurrence(z, x, h, offsets=off)  # no states at all
        d3.recurrence_backward(x, z, x, x, dz, dx, offsets=off)
        assert untouched(h, hb) and untouched(dz, zb) and untouched(dx, xb)
    d3.device_status()
