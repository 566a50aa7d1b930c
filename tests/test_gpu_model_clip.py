"""The norm over all gradients and their clipping against float64 forms.

The norm: squares are summed in fp32 over at most 32 values a thread (16 additions
deep in the worst order: 32 units of 2^-24 relative, all terms positive) and then in
fp64; its root halves that and is rounded once."""
import math

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import TINY, TYPES, U, check, dev, host, out, untouched

pytestmark = pytest.mark.gpu

NORM = 18 * 2.0 ** -24


def workspace():
    return d3.alloc_workspace(d3.grad_norm_workspace_size()).fill_(255)


def norm_ref(ts):
    return math.sqrt(sum(math.fsum((host(t).ravel() ** 2).tolist()) for t in ts))


def factor(norm, max_norm):
    """The factor as 32 bits give it."""
    n = np.float32(norm)
    return min(np.float32(1), np.float32(max_norm) / (n + np.float32(1e-6)))


def make(rng, sizes, scale=1.0):
    """Tensors of every type, matrices with pitches and odd bases among them."""
    ts = []
    for i, (rows, cols) in enumerate(sizes):
        pad, shift = ((0, 0), (3, 1), (8, 0), (0, 3))[i % 4]
        t = dev(scale * rng.standard_normal((rows, cols)), TYPES[i // 2 % 3], pad, shift)
        ts.append(t[0] if rows == 1 else t)
    return ts


SIZES = [[(1, 1)], [(1, 7), (3, 5), (1, 100)], [(64, 64), (1, 64), (33, 1000), (1, 4096), (300, 129), (2, 2)],
         [(700, 900), (5, 16385), (1, 200000), (16384, 3), (1, 1), (40, 8192), (129, 513)],
         [(1 + i % 5, 1 + 37 * i % 700) for i in range(40)], [(1 + i % 3, 1 + i % 50) for i in range(1000)]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[-1][1]}")
def test_norm_and_clip(cuda_lib, sizes):
    rng = np.random.default_rng(len(sizes))
    ts = make(rng, sizes)
    want = norm_ref(ts)
    norm = torch.zeros(1, device="cuda")
    d3.grad_norm(ts, norm, ws=workspace())
    check(host(norm), [want], NORM * want, "norm")
    before = [t.clone() for t in ts]
    for max_norm in (0.5 * want, 2 * want, math.inf, 0.0):
        n2 = torch.zeros((), device="cuda")
        outs = [out(*(t.shape if t.dim() == 2 else (1, t.shape[0])), TYPES[i % 3], *((0, 0), (5, 3), (2, 2))[i % 3])
                for i, t in enumerate(ts)]
        views = [o[0] if t.dim() == 2 else o[0][0] for t, o in zip(ts, outs)]
        d3.clip_grad_norm(ts, max_norm, n2, out=views, ws=workspace())
        assert n2 == norm[0] and all(torch.equal(a, b) for a, b in zip(ts, before))
        f = float(factor(host(norm)[0], max_norm))
        for i, (t, v, o) in enumerate(zip(ts, views, outs)):
            w = host(t) * f
            check(host(v), w, np.abs(w) * (2.0 ** -23 + 1.001 * U[TYPES[i % 3]]) + TINY[TYPES[i % 3]], f"out {i}")
            assert untouched(*o)
    d3.clip_grad_norm(ts, 2 * want, norm, ws=workspace())  # nothing to clip
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    d3.clip_grad_norm(ts, 0.5 * want, ws=workspace())
    f = float(factor(host(norm)[0], 0.5 * want))
    for t, b in zip(ts, before):
        assert torch.equal(t, (b.float() * f).to(t.dtype))
    d3.grad_norm(ts, norm, ws=workspace())
    # Each clipped value is off by a rounding of its type.
    assert abs(float(norm) / (0.5 * want) - 1) < 2.0 ** -8 + 1e-5


@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e-19, 1e-10, 1e10, 1e18, 1e19, 1e30, 3e37])
def test_every_finite_size(cuda_lib, scale):
    """Squares beyond fp32's range, alone and beside others."""
    rng = np.random.default_rng(1)
    big = torch.from_numpy(scale * rng.uniform(-1, 1, 3001)).float().cuda()
    half = torch.from_numpy(scale * rng.uniform(-1, 1, (3, 700))).to("cuda").to(torch.bfloat16)
    for ts in ([big], [half], [big, half], [big, torch.ones(5000, device="cuda"), half], [torch.zeros(40000, device="cuda"), big]):
        norm = torch.zeros(1, device="cuda")
        d3.grad_norm(ts, norm, ws=workspace())
        want = norm_ref(ts)
        if want > torch.finfo(torch.float32).max:
            # 3001 values up to 3e37 have a norm of 3e37 sqrt(3001 / 3) = 9.5e38, past fp32's 3.4e38: it reads infinity.
            assert torch.isinf(norm).all()
            continue
        check(host(norm), [want], NORM * want + 2.0 ** -149, "norm")


def test_nan_and_infinity(cuda_lib):
    for bad in (float("nan"), float("inf"), -float("inf")):
        ts = [torch.ones(1000, device="cuda"), torch.ones(7, 9, device="cuda", dtype=torch.bfloat16)]
        ts[1][3, 3] = bad
        norm = torch.zeros(1, device="cuda")
        d3.clip_grad_norm(ts, 1.0, norm, ws=workspace())
        if bad != bad:
            assert torch.isnan(norm).all() and torch.isnan(ts[0]).all()
        else:
            assert torch.isinf(norm).all() and not ts[0].any() and torch.isnan(ts[1][3, 3])


def test_nothing(cuda_lib):
    norm = torch.ones(1, device="cuda")
    for ts in ([], [torch.empty(0, device="cuda"), torch.empty(0, 5, device="cuda"), torch.empty(5, 0, device="cuda")],
               [torch.zeros(3000, device="cuda")]):
        d3.grad_norm(ts, norm.fill_(1), ws=workspace())
        assert norm == 0
        d3.clip_grad_norm(ts, 1.0, norm.fill_(1), ws=workspace())
        assert norm == 0
        d3.clip_grad_norm(ts, 1.0, ws=workspace())


def test_columns_of_one_matrix(cuda_lib):
    """Gradients that interleave in one matrix, clipped in place together."""
    w = torch.randn(50, 96, device="cuda")
    before = w.clone()
    norm = torch.empty(1, device="cuda")
    d3.clip_grad_norm([w[:, :32], w[:, 64:], w[:, 32:64]], 1.0, norm, ws=workspace())
    assert torch.equal(w, before * float(factor(host(norm)[0], 1.0)))


def test_more_than_32_bits_of_elements(cuda_lib):
    n = (1 << 32) + 77
    t = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(2.0 ** -16)
    t[-1] = 3.0
    norm = torch.empty(1, device="cuda")
    d3.clip_grad_norm([t], 1.0, norm, ws=workspace())
    want = math.sqrt((n - 1) * 2.0 ** -32 + 9.0)
    check(host(norm), [want], NORM * want, "norm")
    f = torch.tensor(factor(host(norm)[0], 1.0))
    assert t[-1] == (3.0 * f).to(torch.bfloat16) and (t[:-1] == (2.0 ** -16 * f).to(torch.bfloat16)).all()


def test_equal_bits_on_other_streams_and_in_a_graph(cuda_lib):
    rng = np.random.default_rng(3)
    ts = make(rng, SIZES[3])
    ws, norm = workspace(), torch.zeros(1, device="cuda")
    outs = [torch.empty_like(t) for t in ts]
    d3.clip_grad_norm(ts, 1.0, norm, out=outs, ws=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again, n2 = [torch.empty_like(t) for t in ts], torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        d3.clip_grad_norm(ts, 1.0, n2, out=again, ws=ws)
    s.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(outs, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d3.clip_grad_norm(ts, 1.0, n2, out=again, ws=ws)
    for k in (1.0, 0.25):
        for t in ts:
            t.mul_(k)
        g.replay()
        d3.clip_grad_norm(ts, 1.0, norm, out=outs, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(outs, again))


def test_no_limit_clips_nothing(cuda_lib):
    """A max_norm of infinity leaves gradients as they are whose norm is infinite or NaN, too."""
    for value in (3e38, float("inf"), float("nan")):
        for n in (1000, 3000000):  # one launch, and several
            ts = [torch.full((n,), 1.0, device="cuda"), torch.ones(7, 9, device="cuda", dtype=torch.bfloat16)]
            ts[0][:5] = value
            before, norm = [t.clone() for t in ts], torch.zeros(1, device="cuda")
            outs = [torch.zeros_like(ts[0], dtype=torch.float32), torch.zeros_like(ts[1], dtype=torch.float32)]
            d3.clip_grad_norm(ts, math.inf, norm, out=outs, ws=workspace())
            d3.clip_grad_norm(ts, math.inf, norm, ws=workspace())
            assert not torch.isfinite(norm).any()
            for t, b, o in zip(ts, before, outs):
                assert torch.equal(t.nan_to_num(7), b.nan_to_num(7)) and torch.equal(o.nan_to_num(7), b.float().nan_to_num(7))
