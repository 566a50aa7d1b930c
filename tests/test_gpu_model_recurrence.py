"""The gated recurrence and its gradient against float64 forms.

Bounds.  A state takes one step h + w (q - p) at a time, or the same through
composed maps.  w is off by at most 5 units of 2^-23 relative (the exponential's
argument by half a unit times |z| log2 e <= 30, two approximations of 2 units and a
product: for |z| <= 20 that is 20 units of w itself, and w |z| < 0.3 brings it
under 8 of the state), the difference, the product and the sum by one each, and a
composition by as many again, so that a step is off by at most 32 units of
|h_{t-1}| + |x_t|; what a step is off decays with the state (`err` of the reference).
A factor that spans n rows is composed of min(n, 39) others at most (a thread's rows, a
channel's lanes, a cluster's blocks), each within 3 units of itself, and what it carries
has 32 n units in the bound: n terms |h_k| that decay alike.
"""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _model_ref import (TINY, TYPES, U, check, dev, host, numbers, out, recurrence_grad_ref, recurrence_ref, untouched)

pytestmark = pytest.mark.gpu

UNIT = 32 * 2.0 ** -23

# tokens, channels, offsets (None: one sequence)
CASES = [(1, 1, None), (1, 64, None), (7, 33, [0, 3, 7]), (64, 96, list(range(65))), (65, 64, [0, 0, 1, 1, 64, 65, 65]),
         (130, 5, [0, 60, 130]), (1000, 2047, [0, 1, 9, 500, 500, 990, 1000]), (2500, 66, None), (700, 40, [3, 10, 600]),
         (3000, 8, [0, 1000, 1001, 2000, 2999]), (513, 128, None),
         # Long enough for whole boxes of rows: a part of a tile, several tiles, a start and an end inside a box.
         (9000, 72, [5, 77, 4000, 4000, 8989]), (4500, 520, None),
         (33000, 8, [0, 16500, 33000])]


def offsets_of(tokens, offsets):
    return [0, tokens] if offsets is None else offsets


def make(rng, tokens, channels, n, dtype, pad, shift):
    z = 3 * rng.standard_normal((tokens, channels)) + 6 * (rng.random(channels) < 0.5)
    z[rng.random((tokens, channels)) < 0.01] = -np.inf
    z[rng.random((tokens, channels)) < 0.01] = np.inf
    mat = lambda a: dev(a, dtype, pad, shift)  # noqa: E731
    state = lambda: torch.from_numpy(rng.standard_normal((n, channels))).float().cuda()  # noqa: E731
    return mat(z), mat(rng.standard_normal((tokens, channels))), state


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,channels,offsets", CASES)
def test_recurrence(cuda_lib, dtype, tokens, channels, offsets):
    rng = np.random.default_rng(tokens + channels)
    seqs = offsets_of(tokens, offsets)
    n, off = len(seqs) - 1, None if offsets is None else numbers(offsets, 32)
    rows = np.arange(tokens)
    rows = rows[(rows >= seqs[0]) & (rows < seqs[-1])]
    for pad, shift, states in ((0, 0, False), (0, 0, True), (3, 1, True), (2, 2, False)):
        z, x, state = make(rng, tokens, channels, n, dtype, pad, shift)
        first = state() if states else None
        last = torch.full((n, channels), 9.0, device="cuda") if states else None
        h, buf = out(tokens, channels, dtype, pad, shift)
        d3.recurrence(z, x, h, offsets=off, first=first, last=last)
        want, want_last, err, last_err = recurrence_ref(host(z), host(x), seqs, host(first) if states else None)
        tol = UNIT * err + 1.001 * U[dtype] * np.abs(want) + TINY[dtype]
        check(host(h)[rows], want[rows], tol[rows], "h")
        outside = np.setdiff1d(np.arange(tokens), rows)
        assert untouched(h, buf) and (host(h)[outside] == 7.0).all()
        if states:
            check(host(last), want_last, UNIT * last_err, "last")
            d3.recurrence(z, x, x, offsets=off, first=first, last=first)  # in place
            assert torch.equal(x[rows], h[rows]) and torch.equal(first, last)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,channels,offsets", CASES)
def test_recurrence_backward(cuda_lib, dtype, tokens, channels, offsets):
    rng = np.random.default_rng(tokens + channels)
    seqs = offsets_of(tokens, offsets)
    n, off = len(seqs) - 1, None if offsets is None else numbers(offsets, 32)
    rows = np.arange(tokens)
    rows = rows[(rows >= seqs[0]) & (rows < seqs[-1])]
    for pad, shift, states in ((0, 0, False), (0, 0, True), (3, 1, True), (2, 2, False)):
        z, x, state = make(rng, tokens, channels, n, dtype, pad, shift)
        h, dh = (dev(rng.standard_normal((tokens, channels)), dtype, pad, shift) for _ in range(2))
        first, dlast = (state() if states else None for _ in range(2))
        dfirst = torch.full((n, channels), 9.0, device="cuda") if states else None
        dz, zbuf = out(tokens, channels, dtype, pad, shift)
        dx, xbuf = out(tokens, channels, dtype, pad, shift)
        d3.recurrence_backward(dh, z, x, h, dz, dx, offsets=off, first=first, dlast=dlast, dfirst=dfirst)
        hz, hx = host(z), host(x)
        wz, wx, wf, err, first_err = recurrence_grad_ref(host(dh), hz, hx, host(h), seqs,
                                                         host(first) if states else None,
                                                         host(dlast) if states else None)
        prev = np.concatenate([np.zeros((1, channels)), host(h)[:-1]])
        if states:
            for i in range(n):
                if seqs[i + 1] > seqs[i]:
                    prev[seqs[i]] = host(first)[i]
        slope = np.exp(-np.abs(hz)) / (1 + np.exp(-np.abs(hz))) ** 2
        # dx = g - s or w g, each within err and a rounding; dz scales that by its factors.
        tx = UNIT * err + 1.001 * U[dtype] * np.abs(wx) + TINY[dtype]
        tz = UNIT * err * (np.abs(prev) + np.abs(hx)) * slope + 1.001 * U[dtype] * np.abs(wz) + TINY[dtype]
        check(host(dx)[rows], wx[rows], tx[rows], "dx")
        check(host(dz)[rows], wz[rows], tz[rows], "dz")
        outside = np.setdiff1d(np.arange(tokens), rows)
        assert untouched(dz, zbuf) and untouched(dx, xbuf)
        assert (host(dz)[outside] == 7.0).all() and (host(dx)[outside] == 7.0).all()
        if states:
            check(host(dfirst), wf, UNIT * first_err, "dfirst")
            d3.recurrence_backward(dh, z, x, h, z, dh, offsets=off, first=first, dlast=dlast, dfirst=dlast)
            assert torch.equal(z[rows], dz[rows]) and torch.equal(dh[rows], dx[rows]) and torch.equal(dlast, dfirst)


@pytest.mark.parametrize("channels", [40, 2048])
def test_gradient_against_differences(cuda_lib, channels):
    """The gradient of sum(c h) + sum(e last) along a direction, against central
    differences of the float64 form."""
    rng = np.random.default_rng(3)
    tokens, seqs = 150, [0, 70, 70, 149]
    z, x = (rng.standard_normal((tokens, channels)) for _ in range(2))
    first = rng.standard_normal((3, channels))
    c, e = rng.standard_normal((tokens, channels)), rng.standard_normal((3, channels))
    c[149:] = 0

    def value(z, x, first):
        h, last, _, _ = recurrence_ref(z, x, seqs, first)
        return float((c * np.nan_to_num(h)).sum() + (e * last).sum())

    t = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    h = torch.zeros(tokens, channels, device="cuda")
    off = numbers(seqs, 32)
    d3.recurrence(t(z), t(x), h, offsets=off, first=t(first))
    dz, dx, dfirst = torch.zeros_like(h), torch.zeros_like(h), torch.zeros(3, channels, device="cuda")
    d3.recurrence_backward(t(c), t(z), t(x), h, dz, dx, offsets=off, first=t(first), dlast=t(e), dfirst=dfirst)
    vz, vx, vf = (rng.standard_normal(a.shape) for a in (z, x, first))
    eps = 1e-5
    num = (value(z + eps * vz, x + eps * vx, first + eps * vf) - value(z - eps * vz, x - eps * vx, first - eps * vf)) / (
        2 * eps)
    terms = [host(dz) * vz, host(dx) * vx, host(dfirst) * vf]
    # The differences are off by eps^2 and by 2^-52 / eps of the sums; the gradients by 32 bits.
    assert abs(sum(float(v.sum()) for v in terms) - num) < 2e-6 * sum(float(np.abs(v).sum()) for v in terms)


def test_a_kept_state_does_not_drift(cuda_lib):
    """Thousands of rows of a gate near 1: the decay is that of 1 - a, not of a rounded a."""
    tokens, channels = 30000, 64
    z = torch.linspace(6, 12, channels, device="cuda").expand(tokens, channels).contiguous()
    x = torch.randn(tokens, channels, device="cuda") + 1
    h = torch.empty_like(x)
    d3.recurrence(z, x, h)
    want, _, err, _ = recurrence_ref(host(z), host(x), [0, tokens], None)
    # A plain sum of roundings of the state: at most (memory) x 2^-24 of it, and some in practice.
    rel = np.abs(host(h) - want)[-1] / np.abs(want[-1])
    a = 1 / (1 + np.exp(-host(z)[0]))
    assert (rel < 4 * np.sqrt(np.minimum(tokens, 1 / (1 - a))) * 2.0 ** -24 + 8 * 2.0 ** -23).all()


def test_many_short_sequences(cuda_lib):
    """More sequences than shared memory keeps offsets of, one token each and more."""
    rng = np.random.default_rng(8)
    for lens in (np.ones(1500, dtype=int), rng.integers(0, 4, 4000)):
        seqs = np.concatenate([[0], np.cumsum(lens)])
        tokens, n, channels = int(seqs[-1]), len(lens), 100
        z, x, state = make(rng, tokens, channels, n, "bf16", 0, 0)
        first, last, off = state(), torch.empty(n, channels, device="cuda"), numbers(seqs, 32)
        h, _ = out(tokens, channels, "bf16")
        d3.recurrence(z, x, h, offsets=off, first=first, last=last)
        want, wl, err, le = recurrence_ref(host(z), host(x), seqs, host(first))
        check(host(h), want, UNIT * err + 1.001 * U["bf16"] * np.abs(want) + TINY["bf16"], "h")
        check(host(last), wl, UNIT * le, "last")
        dz, dx, df = torch.empty_like(h), torch.empty_like(h), torch.empty_like(last)
        d3.recurrence_backward(x, z, x, h, dz, dx, offsets=off, first=first, dlast=last, dfirst=df)
        _, wx, wf, err, fe = recurrence_grad_ref(host(x), host(z), host(x), host(h), seqs, host(first), host(last))
        check(host(dx), wx, UNIT * err + 1.001 * U["bf16"] * np.abs(wx) + TINY["bf16"], "dx")
        check(host(df), wf, UNIT * fe, "dfirst")


def test_decode_matches_a_whole_pass(cuda_lib):
    """Token by token with the state carried along: each h is that of the whole sequences."""
    n, tokens, channels = 5, 12, 130
    z, x = torch.randn(n * tokens, channels, device="cuda") + 2, torch.randn(n * tokens, channels, device="cuda")
    h, last = torch.empty_like(x), torch.empty(n, channels, device="cuda")
    d3.recurrence(z, x, h, offsets=numbers(np.arange(n + 1) * tokens, 32), last=last)
    state, one = torch.zeros(n, channels, device="cuda"), numbers(np.arange(n + 1), 32)
    for t in range(tokens):
        y = torch.empty(n, channels, device="cuda")
        d3.recurrence(z[t::tokens], x[t::tokens], y, offsets=one, first=state, last=state)
        _, _, err, _ = recurrence_ref(host(z), host(x), np.arange(n + 1) * tokens, None)
        check(host(y), host(h[t::tokens]), 2 * UNIT * err[t::tokens], "token by token")
    check(host(state), host(last), 2 * UNIT * err[tokens - 1::tokens], "states")


def test_nan_does_not_pass_a_sequence(cuda_lib):
    for tokens, cut in ((400, 130), (20, 7), (1500, 1100)):
        z, x = torch.zeros(tokens, 66, device="cuda"), torch.ones(tokens, 66, device="cuda")
        x[cut - 1, 3], z[cut - 2, 5] = float("nan"), float("nan")
        x[cut, 8] = float("inf")
        off = numbers([0, cut, tokens], 32)
        h, last = torch.empty_like(x), torch.empty(2, 66, device="cuda")
        d3.recurrence(z, x, h, offsets=off, last=last)
        bad = ~torch.isfinite(h)
        assert not bad[cut:, [i for i in range(66) if i != 8]].any() and bad[cut:, 8].all()
        assert bad[cut - 1, [3, 5]].all() and bad.sum() == 1 + 2 + tokens - cut
        dz, dx = torch.empty_like(x), torch.empty_like(x)
        d3.recurrence_backward(x, z, torch.ones_like(x), torch.ones_like(x), dz, dx, offsets=off)
        bad = ~torch.isfinite(dx)
        assert not bad[cut:, [3, 5]].any() and not bad[:cut, 8].any() and bad[:cut, 3].all()


def test_forgetting_is_exact(cuda_lib):
    """z = -inf takes x whatever the state was, even one that overflowed."""
    x = torch.randn(300, 64, device="cuda")
    z = torch.full_like(x, float("-inf"))
    h = torch.empty_like(x)
    d3.recurrence(z, x, h, first=torch.full((1, 64), 3e38, device="cuda"))
    assert torch.equal(h, x)
    last = torch.empty(1, 64, device="cuda")
    d3.recurrence(-z, x, h, first=x[:1].contiguous(), last=last)
    assert (h == x[:1]).all() and torch.equal(last, x[:1])


def test_no_rows(cuda_lib):
    e = torch.empty(0, 8, device="cuda", dtype=torch.bfloat16)
    first, last = torch.randn(3, 8, device="cuda"), torch.zeros(3, 8, device="cuda")
    off = numbers([0, 0, 0, 0], 32)
    d3.recurrence(e, e, e, offsets=off, first=first, last=last)
    assert torch.equal(first, last)
    d3.recurrence_backward(e, e, e, e, e, e, offsets=off, dlast=first, dfirst=last.zero_())
    assert torch.equal(first, last)
    d3.recurrence(e, e, e, offsets=off, last=last)
    assert not last.any()
    d3.recurrence(e, e, e, offsets=numbers([0], 32))


def test_offsets_past_32_bits(cuda_lib):
    tokens, channels = 270, 64
    big = torch.zeros(tokens, 1 << 24, dtype=torch.bfloat16, device="cuda")
    z, x, h = big[:, :64], big[:, 64:128], big[:, 128:192]
    z.copy_(torch.randn(tokens, 64, device="cuda"))
    x.copy_(torch.randn(tokens, 64, device="cuda"))
    d3.recurrence(z, x, h)
    small = torch.empty(tokens, 64, dtype=torch.bfloat16, device="cuda")
    d3.recurrence(z.contiguous(), x.contiguous(), small)
    assert torch.equal(h, small)
    dz, dx = big[:, 192:256], big[:, 256:320]
    sz, sx = torch.empty_like(small), torch.empty_like(small)
    d3.recurrence_backward(x, z, x, h, dz, dx)
    d3.recurrence_backward(x.contiguous(), z.contiguous(), x.contiguous(), small, sz, sx)
    assert torch.equal(dz, sz) and torch.equal(dx, sx)


def test_offsets_that_do_not_ascend_stay_inside(cuda_lib):
    """Bad offsets: no write outside the rows, and the call ends."""
    for off in ([0, 500, 100, 400], [-5, 900, -7, 2000], [400, 0], [300] * 4, [2 ** 31 - 1, -2 ** 31, 5]):
        h, buf = out(400, 66, "bf16", 2)
        x = torch.ones(400, 66, dtype=torch.bfloat16, device="cuda")
        n = len(off) - 1
        last = torch.full((n + 2, 66), 7.0, device="cuda")
        d3.recurrence(x, x, h, offsets=numbers(off, 32), last=last[1:-1])
        dz, dx = torch.empty_like(x), torch.empty_like(x)
        d3.recurrence_backward(x, x, x, x, dz, dx, offsets=numbers(off, 32), dfirst=last[1:-1])
        assert untouched(h, buf) and (last[0] == 7).all() and (last[-1] == 7).all()


def test_equal_bits_on_other_streams_and_in_a_graph(cuda_lib):
    rng = np.random.default_rng(2)
    tokens, channels = 3000, 512
    z, x, _ = make(rng, tokens, channels, 1, "bf16", 0, 0)
    off = numbers([0, 100, 1700, tokens], 32)
    h, dz, dx = (torch.empty_like(x) for _ in range(3))
    d3.recurrence(z, x, h, offsets=off)
    d3.recurrence_backward(x, z, x, h, dz, dx, offsets=off)
    torch.cuda.synchronize()
    s, (h2, dz2, dx2) = torch.cuda.Stream(), (torch.empty_like(x) for _ in range(3))
    with torch.cuda.stream(s):
        d3.recurrence(z, x, h2, offsets=off)
        d3.recurrence_backward(x, z, x, h2, dz2, dx2, offsets=off)
    s.synchronize()
    assert torch.equal(h, h2) and torch.equal(dz, dz2) and torch.equal(dx, dx2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d3.recurrence(z, x, h2, offsets=off)
        d3.recurrence_backward(x, z, x, h2, dz2, dx2, offsets=off)
    for cuts in ([0, 100, 1700, tokens], [0, 0, 2999, tokens]):
        off.copy_(numbers(cuts, 32))
        g.replay()
        d3.recurrence(z, x, h, offsets=off)
        d3.recurrence_backward(x, z, x, h, dz, dx, offsets=off)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(dz, dz2) and torch.equal(dx, dx2)


def test_two_streams_at_once(cuda_lib):
    """Calls that share nothing but their inputs, side by side."""
    rng = np.random.default_rng(4)
    z, x, _ = make(rng, 6000, 512, 1, "bf16", 0, 0)
    want, wz, wx = (torch.empty_like(x) for _ in range(3))
    d3.recurrence(z, x, want)
    d3.recurrence_backward(x, z, x, want, wz, wx)
    outs = [[torch.empty_like(x) for _ in range(3)] for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (h, dz, dx) in zip(streams, outs):
            with torch.cuda.stream(s):
                d3.recurrence(z, x, h)
                d3.recurrence_backward(x, z, x, h, dz, dx)
    torch.cuda.synchronize()
    for h, dz, dx in outs:
        assert torch.equal(h, want) and torch.equal(dz, wz) and torch.equal(dx, wx)
    d3.device_status()


@pytest.mark.parametrize("dtype,tokens,channels", [("bf16", 700, 128), ("f16", 9000, 64), ("f32", 300, 33)])
def test_states_and_places_in_every_combination(cuda_lib, dtype, tokens, channels):
    """Each state alone, and each result in the place of each input."""
    rng = np.random.default_rng(tokens)
    seqs = [0, tokens // 3, tokens // 3, tokens - 1]
    off = numbers(seqs, 32)
    z, x, state = make(rng, tokens, channels, 3, dtype, 0, 0)
    z.clamp_(-5, 5)
    first, dlast, zero = state(), state(), torch.zeros(3, channels, device="cuda")
    h0, last0, h1, last1 = torch.zeros_like(x), torch.empty_like(first), torch.zeros_like(x), torch.empty_like(first)
    d3.recurrence(z, x, h0, offsets=off, first=first, last=last0)
    d3.recurrence(z, x, h1, offsets=off, first=zero, last=last1)
    for f, want, end in ((first, h0, last0), (None, h1, last1)):
        for ask in (False, True):
            for place in ("z", "x", "new"):
                zi, xi = z.clone(), x.clone()
                h = {"z": zi, "x": xi, "new": torch.empty_like(x)}[place]
                last = torch.empty_like(first) if ask else None
                d3.recurrence(zi, xi, h, offsets=off, first=f, last=last)
                assert torch.equal(h[:-1], want[:-1]) and (not ask or torch.equal(last, end))
    dh = dev(rng.standard_normal((tokens, channels)), dtype)
    for f, dl in ((first, dlast), (first, None), (None, dlast), (None, None)):
        dz0, dx0, df0 = torch.zeros_like(x), torch.zeros_like(x), torch.empty_like(first)
        d3.recurrence_backward(dh, z, x, h0, dz0, dx0, offsets=off, first=zero if f is None else f,
                               dlast=zero if dl is None else dl, dfirst=df0)
        for ask in (False, True):
            for pz, px in (("z", "x"), ("x", "z"), ("dh", "z"), ("x", "dh"), ("new", "x")):
                t = {"z": z.clone(), "x": x.clone(), "dh": dh.clone(), "new": torch.empty_like(x)}
                df = torch.empty_like(first) if ask else None
                d3.recurrence_backward(t["dh"], t["z"], t["x"], h0, t[pz], t[px], offsets=off, first=f, dlast=dl, dfirst=df)
                assert torch.equal(t[pz][:-1], dz0[:-1]) and torch.equal(t[px][:-1], dx0[:-1])
                assert not ask or torch.equal(df, df0)


# Short calls: each on both sides of one and of two rows a thread, sequences of one row, of
# several and of none; and channels whose tiles take clusters of 3, 5, 7 and more blocks.
SHORT = [(1, 4096, 1), (5, 4096, 5), (64, 4096, 64), (65, 4096, 65), (128, 4096, 100), (129, 4096, 129), (30, 4096, 3),
         (16, 1024, 16), (300, 1024, 300), (33, 520, 33), (17, 4096, 1), (32, 4100, 2), (70, 1023, 70), (9, 66, 20)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,channels,n", SHORT + [(2600, 2560, 2), (1500, 1536, 1), (2100, 4864, 3), (900, 700, 1)])
def test_short_calls_and_clusters_of_every_size(cuda_lib, dtype, tokens, channels, n):
    rng = np.random.default_rng(tokens * n)
    cuts = np.sort(rng.integers(0, tokens + 1, n - 1)) if n < tokens else np.arange(1, n).clip(max=tokens)
    seqs = np.concatenate([[0], cuts, [tokens]])
    off = numbers(seqs, 32)
    for states in (True, False):
        z, x, state = make(rng, tokens, channels, n, dtype, 0, 0)
        h, dh = dev(rng.standard_normal((tokens, channels)), dtype), dev(rng.standard_normal((tokens, channels)), dtype)
        first, dlast = (state(), state()) if states else (None, None)
        last, dfirst = (torch.empty(n, channels, device="cuda") for _ in range(2)) if states else (None, None)
        y, dz, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        d3.recurrence(z, x, y, offsets=off, first=first, last=last)
        want, want_last, err, last_err = recurrence_ref(host(z), host(x), seqs, host(first) if states else None)
        check(host(y), want, UNIT * err + 1.001 * U[dtype] * np.abs(want) + TINY[dtype], "h")
        if states:
            check(host(last), want_last, UNIT * last_err, "last")
        d3.recurrence_backward(dh, z, x, h, dz, dx, offsets=off, first=first, dlast=dlast, dfirst=dfirst)
        hz, hx, prev = host(z), host(x), np.concatenate([np.zeros((1, channels)), host(h)[:-1]])
        wz, wx, wf, err, first_err = recurrence_grad_ref(host(dh), hz, hx, host(h), seqs, host(first) if states else None,
                                                         host(dlast) if states else None)
        for i in range(n):
            if seqs[i + 1] > seqs[i]:
                prev[seqs[i]] = host(first)[i] if states else 0.0
        slope = np.exp(-np.abs(hz)) / (1 + np.exp(-np.abs(hz))) ** 2
        check(host(dx), wx, UNIT * err + 1.001 * U[dtype] * np.abs(wx) + TINY[dtype], "dx")
        check(host(dz), wz, UNIT * err * (np.abs(prev) + np.abs(hx)) * slope + 1.001 * U[dtype] * np.abs(wz) + TINY[dtype],
              "dz")
        if states:
            check(host(dfirst), wf, UNIT * first_err, "dfirst")
