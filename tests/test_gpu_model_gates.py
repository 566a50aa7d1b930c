"""The recurrence's gates far from 0, each relative to itself.

With e = z log2 e + 1, |e| < 128: the constant is off by 2^-25 of itself and the sum is
rounded once at 2^-18, so e is off by 2^-18 + 2^-18 and the exponential by ln 2 times that,
5.3e-6; the exponential and the reciprocal by 2^-22 and 2^-23, and a product by 2^-24:
5.8e-6 for a row's h, one more product of a and 1 - a and two of the gradient for dz.
a may be 0 below 2^-126 (z < -87.33), and 1 - a below 2^-125 (z > 86.64).
"""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import _gates, host, numbers

pytestmark = pytest.mark.gpu

A, DZ = 6e-6, 7e-6


def least(v, bound):
    """What a gate of v may be off by where it may be flushed."""
    return np.where(v < 1.001 * bound, v, 0.0)


def rows_of(lo, hi, tokens, channels):
    z = torch.linspace(lo, hi, tokens * channels, dtype=torch.float64).float().view(tokens, channels)
    return z[:, torch.randperm(channels, generator=torch.Generator().manual_seed(1))].contiguous().cuda()


# Rows a thread of one and of several, boxes and cells, channels by four, two and one.
SHAPES = [(1, 4096), (20, 64), (700, 128), (3000, 33), (1100, 2048), (2100, 66)]


@pytest.mark.parametrize("lo,hi", [(-87.3, -69.0), (-100.0, -87.0), (60.0, 87.0)])
@pytest.mark.parametrize("tokens,channels", SHAPES)
def test_far_gates_keep_their_digits(cuda_lib, tokens, channels, lo, hi):
    """Sequences of one row from a state of 2^100: h is a and dz is a (1 - a), scaled."""
    z = rows_of(lo, hi, tokens, channels)
    off, big = numbers(np.arange(tokens + 1), 32), 2.0 ** 100
    first, x = torch.full((tokens, channels), big, device="cuda"), torch.zeros(tokens, channels, device="cuda")
    h, last, dz, dx = (torch.empty_like(z) for _ in range(4))
    d3.recurrence(z, x, h, offsets=off, first=first, last=last)
    a, na = _gates(host(z))
    la, lna = least(a, 2.0 ** -126), least(na, 2.0 ** -125)
    assert (np.abs(host(h) / big - a) <= A * a + la).all() and torch.equal(h, last)
    d3.recurrence_backward(torch.ones_like(z), z, x, h, dz, dx, offsets=off, first=first)
    want = a * na
    assert (np.abs(host(dz) / big - want) <= DZ * want + la + lna).all()
    assert (np.abs(host(dx) - na) <= A * na + lna).all()


def test_a_far_gate_inside_a_sequence(cuda_lib):
    """Rows that keep the state around one that all but forgets it: the maps of threads,
    lanes and blocks carry its small factor."""
    for tokens, channels in ((600, 128), (5000, 64), (900, 33)):
        for at in (0, 1, tokens // 2, tokens - 2):
            z = torch.full((tokens, channels), float("inf"), device="cuda")
            z[at] = torch.linspace(-87.2, -70, channels, device="cuda")
            h, x = torch.empty_like(z), torch.zeros_like(z)
            d3.recurrence(z, x, h, first=torch.full((1, channels), 2.0 ** 100, device="cuda"))
            want = _gates(host(z[at]))[0] * 2.0 ** 100
            assert (h[:at] == 2.0 ** 100).all() and (np.abs(host(h[at:]) - want) <= 2 * A * want).all()
