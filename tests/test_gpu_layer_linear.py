"""The linear layer and its gradient against float64 forms: token counts from
one, odd widths, pitches and bases, saved activations in 16 and 8 bits."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _harness import torch_dtype
from _layer_ref import (ACTS, TINY, U, act_ref, check, check_packed, dact_ref, linear_grad_ref, linear_ref, sum_bound,
                        values_ref)
from test_gpu_layer_norm import dev, host, out, packed, untouched

pytestmark = pytest.mark.gpu

ACT = dict(none=d3.ACT_NONE, relu=d3.ACT_RELU, gelu=d3.ACT_GELU, silu=d3.ACT_SILU)
#: Largest slope of the activations (gelu's is 1.13), and the error of the
#: fp32 exponential and division in them, relative to |z|: exp's argument is
#: rounded at up to 8 |z| and the rest is a few 2^-24.
SLOPE, ACT_ERR = 1.13, 2.0 ** -18

SIZES = [  # tokens, in, out
    (1, 1, 1), (1, 64, 128), (2, 7, 33), (16, 256, 100), (17, 72, 264), (33, 130, 31), (64, 512, 256), (65, 65, 129),
    (127, 1000, 96), (128, 64, 512), (129, 2047, 130), (300, 320, 257), (513, 200, 1030), (1, 4096, 1001),
    (700, 1032, 776),
    # several large tiles a cluster, in one product of the layer or another; odd widths with them
    (2100, 72, 2050), (130, 2080, 2201), (257, 2303, 2048), (4100, 40, 300),
    # a few tokens through many rows
    (1, 520, 2100), (2, 8, 2048), (3, 264, 2077), (4, 1032, 2049), (5, 1032, 2049)]


def ws_for(fn, t, k, n, dtype, strided):
    return d3.alloc_workspace(fn(t, k, n, dtype=torch_dtype(dtype), strided=strided))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,k,n", SIZES)
@pytest.mark.parametrize("form", ["bare", "all16", "all8", "strided"])
def test_linear(cuda_lib, dtype, t, k, n, form):
    rng = np.random.default_rng(t * 31 + k * 7 + n)
    act = ACTS[(t + k + n + len(form)) % 4] if form != "bare" else "none"
    pad, shift = (3, 5) if form == "strided" else (0, 0)
    x, w = dev(rng, t, k, dtype, 1.0, pad, shift), dev(rng, n, k, dtype, k ** -0.5, pad, shift)
    full = form != "bare"
    b = torch.from_numpy(rng.standard_normal(n)).to("cuda").to(torch_dtype("f32" if form == "all8" else dtype)) \
        if full else None
    r = dev(rng, t, n, dtype, 1.0, pad, shift) if full else None
    y, ybuf = out(t, n, dtype, pad, shift)
    z16, zbuf = out(t, n, dtype, pad, shift) if form in ("all16", "strided") else (None, None)
    z8, y8 = (packed(t, n), packed(t, n, 7)) if form == "all8" else (None, None)
    ws = ws_for(d3.linear_workspace_size, t, k, n, dtype, form == "strided")
    d3.linear(x, w, y, bias=b, residual=r, act=ACT[act], z=z8 if z8 is not None else z16, y8=y8, ws=ws)
    d3.device_status()
    hx, hw = host(x), host(w)
    zr, yr = linear_ref(hx, hw, None if b is None else host(b), act, None if r is None else host(r))
    zerr = (np.abs(hx) @ np.abs(hw).T) * sum_bound(k) + np.abs(zr) * 2.0 ** -23
    yerr = zerr * SLOPE + np.abs(zr) * (ACT_ERR if act in ("gelu", "silu") else 0) + np.abs(yr) * 2.0 ** -23
    check(host(y), yr, yerr + (np.abs(yr) + yerr) * U[dtype] + TINY[dtype], f"y ({act})")
    assert untouched(y, ybuf)
    if z16 is not None:
        check(host(z16), zr, zerr + (np.abs(zr) + zerr) * U[dtype] + TINY[dtype], "z")
        assert untouched(z16, zbuf)
    if z8 is not None:
        check_packed(z8.codes.cpu(), z8.scales.cpu(), zr, zerr, "z8")
        check_packed(y8.codes.cpu(), y8.scales.cpu(), yr, yerr, "y8")
        nb = -(-n // 32)  # the spare columns of y8's pitch
        assert bool((y8.codes.as_strided((t, 7), (n + 7, 1), n) == 99).all())
        assert bool((y8.scales.as_strided((t, 7), (nb + 7, 1), nb) == 99).all())


def pack_host(p):
    return values_ref(p.codes.cpu().numpy().astype(np.int64), p.scales.cpu().numpy().astype(np.int64))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,k,n", SIZES)
@pytest.mark.parametrize("form", ["bare", "all16", "all8", "strided"])
def test_linear_backward(cuda_lib, dtype, t, k, n, form):
    rng = np.random.default_rng(t * 13 + k * 5 + n)
    act = ACTS[(t + k + n + len(form)) % 4] if form != "bare" else "none"
    pad, shift = (3, 5) if form == "strided" else (0, 0)
    x, w = dev(rng, t, k, dtype, 1.0, pad, shift), dev(rng, n, k, dtype, k ** -0.5, pad, shift)
    dy, z = dev(rng, t, n, dtype, 0.1, pad, shift), dev(rng, t, n, dtype, 1.5, pad, shift)
    hx, hw, hdy, hz = host(x), host(w), host(dy), host(z)
    if form == "all8":
        x8, z8 = packed(t, k), packed(t, n, 5)
        d3.pack8(x, x8)
        d3.pack8(z, z8)
        x, z, hx, hz = x8, z8, pack_host(x8), pack_host(z8)
        if dtype == "f16":  # a block's value in fp16
            hx = torch.from_numpy(hx).half().double().numpy()
    grad = ("f32", "bf16", "f16")[(t + n + len(form)) % 3]
    dx, dxbuf = out(t, k, dtype, pad, shift)
    dw, dwbuf = out(n, k, grad, pad, shift)
    db = torch.full((n,), 3.0, device="cuda")
    ws = ws_for(d3.linear_backward_workspace_size, t, k, n, dtype, form == "strided")
    args = dict(act=ACT[act], z=None if act == "none" else z, ws=ws)
    d3.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, **args)
    d3.device_status()
    dz, dxr, dwr, dbr = linear_grad_ref(hdy, hx, hw, act, hz)
    derr = np.abs(hdy) * (1 + np.abs(hz)) * (ACT_ERR if act in ("gelu", "silu") else 0)  # of the unrounded dz
    rerr = derr + (0 if act == "none" else np.abs(dz) * U[dtype] * 1.001 + TINY[dtype])  # of the rounded one
    az = np.abs(dz) + rerr
    for name, got, want, e, dt in (
            ("dx", dx, dxr, rerr @ np.abs(hw) + (az @ np.abs(hw)) * sum_bound(n), dtype),
            ("dw", dw, dwr, rerr.T @ np.abs(hx) + (az.T @ np.abs(hx)) * sum_bound(t), grad)):
        check(host(got), want, e + (np.abs(want) + e) * U[dt] + TINY[dt], f"{name} ({act})")
    check(host(db), dbr, derr.sum(0) + np.abs(dz).sum(0) * sum_bound(min(t, 700)), "db")
    assert untouched(dx, dxbuf) and untouched(dw, dwbuf)
    first, fdb, fdx = dw.clone(), db.clone(), dx.clone()
    d3.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, **args)
    assert torch.equal(dw, first) and torch.equal(db, fdb) and torch.equal(dx, fdx), "the same bits every call"
    d3.linear_backward(dy, x, w, dw=dw, db=db, accumulate=True, **args)  # the same sums again on top
    assert torch.equal(db, fdb + fdb)
    e = rerr.T @ np.abs(hx) + (az.T @ np.abs(hx)) * sum_bound(t)
    # the stored dw was rounded once; the new sum is rounded once more
    check(host(dw), host(first) + dwr, e + (np.abs(host(first) + dwr) + e) * U[grad] * 1.01 + TINY[grad], "dw +=")


def test_linear_backward_against_differences(cuda_lib):
    rng = np.random.default_rng(4)
    for act in ("gelu", "silu"):
        x, w, dy = dev(rng, 3, 16, "bf16"), dev(rng, 8, 16, "bf16", 0.3), dev(rng, 3, 8, "bf16")
        b = torch.from_numpy(rng.standard_normal(8)).float().cuda()
        y, z = torch.empty(3, 8, dtype=torch.bfloat16, device="cuda"), d3.alloc_packed8(3, 8)
        z16 = torch.empty_like(y)
        d3.linear(x, w, y, bias=b, act=ACT[act], z=z16)
        dx, dw, db = torch.empty_like(x), torch.empty(8, 16, device="cuda"), torch.empty(8, device="cuda")
        ws = ws_for(d3.linear_backward_workspace_size, 3, 16, 8, "bf16", False)
        d3.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, act=ACT[act], z=z16, ws=ws)
        hx, hw, hb, c = host(x), host(w), host(b), host(dy)
        loss = lambda a_, w_, b_: float((linear_ref(a_, w_, b_, act, None)[1] * c).sum())  # noqa: E731
        # z is kept in bf16 (relative 2^-8, slope of act' at most 1.2) and dz is rounded to it (2^-8)
        dzerr = np.abs(c) * ((np.abs(hx @ hw.T + hb)) * 1.2 + 1.13) * 2.0 ** -8
        e = 1e-5
        for got, arg, tol in ((dx, 0, dzerr @ np.abs(hw) + np.abs(host(dx)) * 2.0 ** -8),
                              (dw, 1, dzerr.T @ np.abs(hx)), (db, 2, dzerr.sum(0))):
            base = [hx, hw, hb]
            for i in np.ndindex(base[arg].shape):
                d = np.zeros_like(base[arg])
                d[i] = e
                up, dn = list(base), list(base)
                up[arg], dn[arg] = base[arg] + d, base[arg] - d
                diff = (loss(*up) - loss(*dn)) / (2 * e)
                assert abs(diff - host(got)[i]) <= tol[i] + 1e-6, (act, arg, i)
        del z


def test_linear_in_place_residual_and_special_values(cuda_lib):
    rng = np.random.default_rng(6)
    x, w, r = dev(rng, 40, 128, "bf16"), dev(rng, 64, 128, "bf16", 0.1), dev(rng, 40, 64, "bf16")
    y, y2 = torch.empty_like(r), r.clone()
    d3.linear(x, w, y, residual=r, act=d3.ACT_GELU)
    d3.linear(x, w, y2, residual=y2, act=d3.ACT_GELU)
    assert torch.equal(y, y2)
    # NaN and infinity stay in their own token (forward, dx) or feature (dw)
    x[3, 5], x[7, 0] = float("nan"), float("inf")
    z8 = d3.alloc_packed8(40, 64)
    d3.linear(x, w, y2, residual=r, act=d3.ACT_GELU, z=z8)
    assert torch.isnan(y2[3]).all() and (z8.scales[3] == 255).all()
    rows = [i for i in range(40) if i not in (3, 7)]
    assert torch.equal(y2[rows], y[rows]) and not torch.isfinite(y2[7]).all()
    dw = torch.empty(64, 128, device="cuda")
    d3.linear_backward(y, x, w, dw=dw)
    cols = [i for i in range(128) if i not in (0, 5)]
    assert torch.isnan(dw[:, 5]).all() and torch.isfinite(dw[:, cols]).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_activation_far_out(cuda_lib, act):
    """Values where exp overflows or the sigmoid is 0 or 1: exact limits, no NaN."""
    v = torch.tensor([0.0, -0.0, 1e4, -1e4, 88.0, -88.0, 200.0, -200.0, 3e38, -3e38, 1e20, -1e20], dtype=torch.bfloat16,
                     device="cuda")
    n = v.numel()
    x, eye = v[:, None].contiguous(), torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    d3.linear(x, eye, y, act=ACT[act], ws=ws_for(d3.linear_workspace_size, n, 1, 1, "bf16", True))
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(host(v) > 80, host(v), np.where(host(v) < -80, 0.0, 0.0))
    check(host(y)[:, 0], want, 1e-30, "act")
    dz = torch.empty(n, 1, device="cuda")
    ws = ws_for(d3.linear_backward_workspace_size, n, 1, 1, "bf16", True)
    dx = torch.empty_like(x)
    d3.linear_backward(torch.ones_like(x), None, eye, dx=dx, act=ACT[act], z=x, ws=ws)
    slope = np.where(host(v) > 80, 1.0, np.where(host(v) < -80, 0.0, 0.0 if act == "relu" else 0.5))
    check(host(dx)[:, 0], slope, 1e-30, "act'")
    del dz


def test_linear_no_tokens(cuda_lib):
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = torch.ones(48, 40, dtype=torch.bfloat16, device="cuda")
    d3.linear(e(40), w, e(48), act=d3.ACT_SILU, z=d3.alloc_packed8(0, 48))
    for grad in (torch.float32, torch.bfloat16):
        dw, db = torch.full((48, 40), 2.0, dtype=grad, device="cuda"), torch.full((48,), 2.0, device="cuda")
        d3.linear_backward(e(48), e(40), w, dx=e(40), dw=dw, db=db, accumulate=True)
        assert bool((dw == 2.0).all()) and bool((db == 2.0).all())
        d3.linear_backward(e(48), e(40), w, dx=e(40), dw=dw, db=db)
        assert bool((dw == 0.0).all()) and bool((db == 0.0).all())


def test_linear_parts_match_the_whole(cuda_lib):
    """Each gradient asked for alone, on another stream and in a replayed graph: the same bits."""
    rng = np.random.default_rng(9)
    t, k, n = 200, 264, 328
    x, w, dy, z = (dev(rng, *s, "bf16") for s in ((t, k), (n, k), (t, n), (t, n)))
    ws = ws_for(d3.linear_backward_workspace_size, t, k, n, "bf16", False)
    new = lambda: (torch.zeros_like(x), torch.zeros(n, k, device="cuda"), torch.zeros(n, device="cuda"))  # noqa: E731
    dx, dw, db = new()
    kw = dict(act=d3.ACT_SILU, z=z, ws=ws)
    d3.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, **kw)
    a, b, c = new()
    d3.linear_backward(dy, None, w, dx=a, **kw)
    d3.linear_backward(dy, x, w, dw=b, **kw)
    d3.linear_backward(dy, None, w, db=c, **kw)
    assert torch.equal(a, dx) and torch.equal(b, dw) and torch.equal(c, db)
    torch.cuda.synchronize()
    a, b, c = new()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    d3.linear_backward(dy, x, w, dx=a, dw=b, db=c, stream=s, **kw)
    s.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dw) and torch.equal(c, db)
    a, b, c = new()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d3.linear_backward(dy, x, w, dx=a, dw=b, db=c, **kw)
    for _ in range(2):
        g.replay()
    assert torch.equal(a, dx) and torch.equal(b, dw) and torch.equal(c, db)
    assert float(np.abs(act_ref("silu", host(z))).max()) > 0 and dact_ref("none", host(z)).all()


@pytest.mark.parametrize("grad,pad", [("f32", 0), ("f32", 1), ("bf16", 0), ("bf16", 3)])
def test_weight_gradient_over_many_tokens(cuda_lib, grad, pad):
    """A 32-bit gradient is summed in pieces over the tokens; written, then added to."""
    t, k, n = 9000, 2080, 2201
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(t, k, generator=g, device="cuda").bfloat16()
    dy = torch.randn(t, n, generator=g, device="cuda").bfloat16()
    w = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    dw, buf = out(n, k, grad, pad)
    ws = ws_for(d3.linear_backward_workspace_size, t, k, n, "bf16", False)
    want, size = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    d3.linear_backward(dy, x, w, dw=dw, ws=ws)
    d3.device_status()
    tol = size * sum_bound(t) + want.abs() * (U[grad] * 1.01)
    assert bool(((dw.double() - want).abs() <= tol).all()) and untouched(dw, buf)
    # 9000 tokens in 3 pieces of at most 64 x 4 accumulations: 2^-23 of a partial sum each, whose
    # root mean square grows to the result's
    if grad == "f32":
        assert float((dw.double() - want).norm() / want.norm()) <= 256 * 2.0 ** -23
    first = dw.clone()
    d3.linear_backward(dy, x, w, dw=dw, ws=ws)
    assert torch.equal(dw, first), "the same bits every call"
    d3.linear_backward(dy, x, w, dw=dw, ws=ws, accumulate=True)
    tol = size * sum_bound(t) + (want.abs() + first.double().abs()) * (U[grad] * 1.01)
    assert bool(((dw.double() - first.double() - want).abs() <= tol).all()) and untouched(dw, buf)


def test_offsets_past_32_bits(cuda_lib):
    """More than 2^31 elements in x's blocks, y, z and dz: the last rows are right."""
    t, k, n = 140_000, 64, 16_384
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(n, k, generator=g, device="cuda").bfloat16() / 8
    y = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    y8 = d3.alloc_packed8(t, n)
    d3.linear(x, w, y, act=d3.ACT_RELU, y8=y8)
    rows = torch.tensor([0, 1, 131_071, 131_072, t - 2, t - 1], device="cuda")
    want = torch.relu(x[rows].double() @ w.double().t())
    size = x[rows].double().abs() @ w.double().abs().t()
    tol = size * sum_bound(k) + want * (U["bf16"] * 1.001)
    assert bool(((y[rows].double() - want).abs() <= tol).all())
    back = torch.empty_like(y)
    d3.unpack8(y8, back)
    step = torch.exp2(y8.scales[rows].double() - 127).repeat_interleave(32, dim=1)
    assert bool(((back[rows].double() - want).abs() <= 0.5 * step + size * sum_bound(k)).all())
    dx = torch.empty_like(x)  # act' of relu from the blocks is 1 where the code is not 0
    ws = ws_for(d3.linear_backward_workspace_size, t, k, n, "bf16", False)
    d3.linear_backward(y, None, w, dx=dx, act=d3.ACT_RELU, z=y8, ws=ws)
    dz = y[rows].double() * (back[rows] > 0)
    tol = (dz.abs() @ w.double().abs()) * sum_bound(n)
    want = dz @ w.double()
    assert bool(((dx[rows].double() - want).abs() <= tol + (want.abs() + tol) * U["bf16"]).all())
    d3.device_status()
