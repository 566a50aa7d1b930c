"""8-bit blocks and the RMS norm (forward and backward) against float64 forms:
odd widths, pitches and bases, every type, special values, refusals aside."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from _harness import torch_dtype
from _layer_ref import TINY, U, check, check_packed, norm_grad_ref, norm_ref, pack_ref, values_ref

pytestmark = pytest.mark.gpu

TYPES = ("f32", "bf16", "f16")


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def dev(rng, rows, cols, dtype, scale=1.0, pad=0, shift=0):
    """A random matrix with `pad` spare columns in its pitch, `shift` elements into its buffer."""
    buf = torch.zeros(rows * (cols + pad) + shift + 8, dtype=torch_dtype(dtype), device="cuda")
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.from_numpy(rng.standard_normal((rows, cols)) * scale))
    return v


def vec(rng, n, dtype):
    return torch.from_numpy(1 + 0.2 * rng.standard_normal(n)).to("cuda").to(torch_dtype(dtype))


def out(rows, cols, dtype, pad=0, shift=0):
    """An output filled with a marker, and its whole buffer."""
    buf = torch.full((rows * (cols + pad) + shift + 8,), 7.0, dtype=torch_dtype(dtype), device="cuda")
    return buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def untouched(v, buf):
    """Nothing outside v's rows was written."""
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
    return bool((buf[keep] == 7.0).all())


def packed(rows, cols, pad=None):
    if pad is None:
        return d3.alloc_packed8(rows, cols)
    nb = -(-cols // 32)
    return d3.Packed8(torch.full((rows, cols + pad), 99, dtype=torch.int8, device="cuda")[:, :cols],
                      torch.full((rows, nb + pad), 99, dtype=torch.uint8, device="cuda")[:, :nb])


SHAPES = [(1, 1), (1, 4096), (3, 31), (2, 32), (5, 33), (7, 100), (4, 1000), (33, 256), (2, 2047), (3, 8200), (300, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack8_is_exact(cuda_lib, dtype, rows, cols):
    rng = np.random.default_rng(rows * 7919 + cols)
    for pad, shift in ((0, 0), (5, 3), (8, 8)):
        x = dev(rng, rows, cols, dtype, pad=pad, shift=shift)
        x *= torch.from_numpy(np.exp2(rng.integers(-12, 12, (rows, 1)).astype(np.float64))).to("cuda").to(x.dtype)
        p = packed(rows, cols, None if pad == 0 else pad)
        d3.pack8(x, p)
        q, b = pack_ref(host(x))
        assert np.array_equal(p.codes.cpu().numpy(), q) and np.array_equal(p.scales.cpu().numpy(), b)
        for to in TYPES:
            v, buf = out(rows, cols, to, pad, shift)
            d3.unpack8(p, v)
            want = torch.from_numpy(values_ref(q, b)).to(v.dtype).to(torch.float64).numpy()
            assert np.array_equal(host(v), want) and untouched(v, buf)


def test_pack8_extremes(cuda_lib):
    rows = [[0.0] * 32, [-0.0] * 31 + [1e-45], [3.4028235e38] + [1.0] * 31, [127.0] * 32, [127.00001] + [0.5] * 31,
            [1.17549435e-38] * 32, [127 * 2.0 ** -127] * 32, [128 * 2.0 ** -127] + [2.0 ** -128] * 31,
            [float("nan")] + [1.0] * 31, [float("-inf")] + [1.0] * 31, [2.5, 3.5, -2.5, 127.0] + [0.5] * 28, [-3.4028235e38, 3.39e38] + [1e38] * 30]
    x = torch.tensor(rows, dtype=torch.float32, device="cuda")
    p = d3.alloc_packed8(len(rows), 32)
    d3.pack8(x, p)
    q, b = pack_ref(host(x))
    assert np.array_equal(p.codes.cpu().numpy(), q) and np.array_equal(p.scales.cpu().numpy(), b)
    v = torch.empty_like(x)
    d3.unpack8(p, v)
    fine = [i for i in range(len(rows)) if i not in (8, 9)]
    assert torch.isnan(v[8:10]).all() and np.array_equal(host(v)[fine], values_ref(q, b)[fine])
    assert torch.isfinite(v[fine]).all()


def norm_slack(cols):
    """Relative error of rstd: half that of the 32-bit sum of squares, and its own few operations."""
    return (cols / 2 + 8) * 2.0 ** -24 if cols < 64 else (64 + 8) * 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + [(2, 16400)])
@pytest.mark.parametrize("form", ["plain", "residual", "packed", "strided"])
def test_rms_norm(cuda_lib, dtype, rows, cols, form):
    rng = np.random.default_rng(rows + 31 * cols)
    pad, shift = (3, 1) if form == "strided" else (0, 0)
    x = dev(rng, rows, cols, dtype, 0.7, pad, shift)
    r = None if form == "plain" else dev(rng, rows, cols, dtype, 2.0, pad, shift)
    w = vec(rng, cols, "f32" if form == "packed" else dtype)
    y, ybuf = out(rows, cols, dtype, pad, shift)
    h, hbuf = out(rows, cols, dtype, pad, shift) if r is not None else (None, None)
    y8 = packed(rows, cols, 3 if form == "strided" else None) if form in ("packed", "strided") else None
    rstd = torch.empty(rows, dtype=torch.float32, device="cuda")
    d3.rms_norm(x, w, y, residual=r, h=h, y8=y8, rstd=rstd, eps=1e-5)
    hr, sr, yr = norm_ref(host(x), None if r is None else host(r), host(w), 1e-5)
    slack = norm_slack(cols)
    check(host(rstd), sr, sr * slack, "rstd")
    # h is rounded to 32 bits before it is used
    err = np.abs(yr) * (slack + 3 * 2.0 ** -24)
    check(host(y), yr, err + np.abs(yr) * U[dtype] * (1 + slack) + TINY[dtype], "y")
    assert untouched(y, ybuf)
    if h is not None:
        check(host(h), hr, np.abs(hr) * (U[dtype] + 2.0 ** -24) + TINY[dtype], "h")
        assert untouched(h, hbuf)
    if y8 is not None:
        check_packed(y8.codes.cpu(), y8.scales.cpu(), yr, err, "y8")


@pytest.mark.parametrize("dtype", TYPES)
def test_rms_norm_in_place_and_packed_only(cuda_lib, dtype):
    rng = np.random.default_rng(5)
    x, r, w = dev(rng, 9, 512, dtype), dev(rng, 9, 512, dtype), vec(rng, 512, dtype)
    y, h, y8 = torch.empty_like(x), torch.empty_like(x), d3.alloc_packed8(9, 512)
    d3.rms_norm(x, w, y, residual=r, h=h, y8=y8)
    r2, y2, only = r.clone(), torch.empty_like(x), d3.alloc_packed8(9, 512)
    d3.rms_norm(x, w, y2, residual=r2, h=r2)          # h over the residual
    d3.rms_norm(x, w, residual=r, y8=only)            # 8-bit output alone
    assert torch.equal(y, y2) and torch.equal(h, r2)
    assert torch.equal(only.codes, y8.codes) and torch.equal(only.scales, y8.scales)
    x2 = x.clone()
    d3.rms_norm(x2, w, x2)                             # y over x
    d3.rms_norm(x, w, y)
    assert torch.equal(x2, y)


def test_rms_norm_special_rows(cuda_lib):
    x = torch.ones(4, 64, device="cuda")
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y, rstd, y8 = torch.empty_like(x), torch.empty(4, device="cuda"), d3.alloc_packed8(4, 64)
    d3.rms_norm(x, torch.ones(64, device="cuda"), y, y8=y8, rstd=rstd, eps=0.0625)
    assert torch.equal(y[0], torch.zeros(64, device="cuda")) and float(rstd[0]) == 4.0
    assert torch.isnan(y[1]).all() and float(rstd[2]) == 0.0 and torch.isnan(y[2, 7])
    assert (y8.scales[1] == 255).all() and y8.scales[2].tolist() == [255, 0]
    check(host(y[3]), np.full(64, 1 / np.sqrt(1.0625)), 2.0 ** -22, "y of an ordinary row beside them")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + [(2, 16400), (1500, 40)])
@pytest.mark.parametrize("strided", [False, True])
def test_rms_norm_backward(cuda_lib, dtype, rows, cols, strided):
    rng = np.random.default_rng(rows * 3 + cols)
    pad, shift = (5, 3) if strided else (0, 0)
    h, dy = dev(rng, rows, cols, dtype, 1.5, pad, shift), dev(rng, rows, cols, dtype, 0.1, pad, shift)
    dh = dev(rng, rows, cols, dtype, 0.1, pad, shift) if (rows + cols) % 2 else None
    w = vec(rng, cols, dtype)
    rstd = torch.from_numpy(1 / np.sqrt((host(h) ** 2).mean(1) + 1e-6)).to("cuda").float()
    dx, buf = out(rows, cols, dtype, pad, shift)
    dw = torch.full((cols,), 3.0, device="cuda")
    ws = d3.alloc_workspace(d3.rms_norm_backward_workspace_size(rows, cols))
    d3.rms_norm_backward(dy, h, w, rstd, dx, dh=dh, dw=dw, ws=ws)
    a = [host(dy), host(h), host(w), host(rstd), None if dh is None else host(dh)]
    dxr, dwr = norm_grad_ref(*a)
    hn = np.abs(a[1] * a[3][:, None])
    mean = (np.abs(a[0] * a[2]) * hn).mean(1, keepdims=True)
    err = (np.abs(a[0] * a[2]) * 4 + hn * mean * (min(cols, 128) + 16)) * a[3][:, None] * 2.0 ** -24
    err = err + (0 if dh is None else np.abs(dxr) * 2.0 ** -23)
    check(host(dx), dxr, err + (np.abs(dxr) + err) * U[dtype] + TINY[dtype], "dx")
    assert untouched(dx, buf)
    tol = (np.abs(a[0]) * hn).sum(0) * (min(rows, 640) + 8) * 2.0 ** -24
    check(host(dw), dwr, tol, "dw")
    first = dw.clone()
    d3.rms_norm_backward(dy, h, w, rstd, dx, dh=dh, dw=dw, ws=ws)
    assert torch.equal(dw, first), "the same call gives the same bits"
    d3.rms_norm_backward(dy, h, w, rstd, dx, dh=dh, dw=dw, ws=ws, accumulate=True)
    assert torch.equal(dw, first + first)
    if dh is not None:  # in place over dh, without dw and its workspace
        keep = dh.clone()
        d3.rms_norm_backward(dy, h, w, rstd, dh, dh=dh)
        assert torch.equal(dh, dx)
        dh.copy_(keep)


def among_nans(rng, rows, cols, dtype, scale, pad, shift):
    """As dev, with NaN in everything that is not the matrix."""
    buf = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.from_numpy(rng.standard_normal((rows, cols)) * scale))
    return v


# Rows misaligned alike are copied ahead through shared memory: enough of them that a block takes several, of every
# number of pieces a thread, and aligned ones too wide for registers.  The last form's results are aligned otherwise.
LONG = [(4000, 250), (4000, 1031), (1500, 2049), (900, 5003), (1300, 5003), (640, 9001), (1100, 8300), (320, 8208), (7, 12001), (9, 301)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", LONG)
@pytest.mark.parametrize("pad,shift,other", [(0, 0, 0), (3, 1, 0), (6, 5, 1)])
def test_rms_norm_of_many_rows(cuda_lib, dtype, rows, cols, pad, shift, other):
    rng = np.random.default_rng(rows + cols + pad)
    x, r = (among_nans(rng, rows, cols, dtype, s, pad, shift) for s in (0.7, 2.0))
    w = vec(rng, cols, dtype)
    slack = norm_slack(cols)
    for res in (None, r):
        y, ybuf = out(rows, cols, dtype, pad, shift + other)
        h, hbuf = out(rows, cols, dtype, pad, shift) if res is not None else (None, None)
        rstd = torch.empty(rows, dtype=torch.float32, device="cuda")
        d3.rms_norm(x, w, y, residual=res, h=h, rstd=rstd, eps=1e-5)
        hr, sr, yr = norm_ref(host(x), None if res is None else host(res), host(w), 1e-5)
        check(host(rstd), sr, sr * slack, "rstd")
        err = np.abs(yr) * (slack + 3 * 2.0 ** -24)
        check(host(y), yr, err + np.abs(yr) * U[dtype] * (1 + slack) + TINY[dtype], "y")
        assert untouched(y, ybuf)
        if h is not None:
            check(host(h), hr, np.abs(hr) * (U[dtype] + 2.0 ** -24) + TINY[dtype], "h")
            assert untouched(h, hbuf)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", LONG)
@pytest.mark.parametrize("pad,shift,other", [(0, 0, 0), (3, 1, 0), (6, 5, 1)])
def test_rms_norm_backward_of_many_rows(cuda_lib, dtype, rows, cols, pad, shift, other):
    rng = np.random.default_rng(rows * 3 + cols + pad)
    h, dy, stream = (among_nans(rng, rows, cols, dtype, s, pad, shift) for s in (1.5, 0.1, 0.1))
    w = vec(rng, cols, dtype)
    rstd = torch.from_numpy(1 / np.sqrt((host(h) ** 2).mean(1) + 1e-6)).to("cuda").float()
    ws = d3.alloc_workspace(d3.rms_norm_backward_workspace_size(rows, cols))
    for dh in (None, stream):
        dx, buf = out(rows, cols, dtype, pad, shift + other)
        dw = torch.full((cols,), 3.0, device="cuda")
        d3.rms_norm_backward(dy, h, w, rstd, dx, dh=dh, dw=dw, ws=ws)
        a = [host(dy), host(h), host(w), host(rstd), None if dh is None else host(dh)]
        dxr, dwr = norm_grad_ref(*a)
        hn = np.abs(a[1] * a[3][:, None])
        mean = (np.abs(a[0] * a[2]) * hn).mean(1, keepdims=True)
        err = (np.abs(a[0] * a[2]) * 4 + hn * mean * (128 + 16)) * a[3][:, None] * 2.0 ** -24
        err = err + (0 if dh is None else np.abs(dxr) * 2.0 ** -23)
        check(host(dx), dxr, err + (np.abs(dxr) + err) * U[dtype] + TINY[dtype], "dx")
        assert untouched(dx, buf)
        check(host(dw), dwr, (np.abs(a[0]) * hn).sum(0) * (min(rows, 640) + 8) * 2.0 ** -24, "dw")
        first = dw.clone()
        d3.rms_norm_backward(dy, h, w, rstd, dx, dh=dh, dw=dw, ws=ws)
        assert torch.equal(dw, first), "the same call gives the same bits"
    same = dx.clone()
    d3.rms_norm_backward(dy, h, w, rstd, stream, dh=stream)  # in place over dh, without dw and its workspace
    if not other:
        assert torch.equal(stream, same)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(300, 2048), (319, 1031), (640, 512), (70, 8192)])
def test_rms_norm_backward_in_place_over_dy(cuda_lib, dtype, rows, cols):
    """dw of few rows is summed beside dx, but not where dx takes dy's place."""
    rng = np.random.default_rng(rows)
    h, dy, w = dev(rng, rows, cols, dtype), dev(rng, rows, cols, dtype), vec(rng, cols, dtype)
    rstd = torch.from_numpy(1 / np.sqrt((host(h) ** 2).mean(1))).to("cuda").float()
    ws = d3.alloc_workspace(d3.rms_norm_backward_workspace_size(rows, cols))
    dx, dw, dw2 = torch.empty_like(dy), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    d3.rms_norm_backward(dy, h, w, rstd, dx, dw=dw, ws=ws)
    hn = np.abs(host(h) * host(rstd)[:, None])
    tol = (np.abs(host(dy)) * hn).sum(0) * (rows + 8) * 2.0 ** -24  # of either sum, in any order
    want = norm_grad_ref(host(dy), host(h), host(w), host(rstd), None)[1]
    check(host(dw), want, tol, "dw")
    d3.rms_norm_backward(dy, h, w, rstd, dy, dw=dw2, ws=ws)
    check(host(dw2), want, tol, "dw in place")
    rel = torch.linalg.vector_norm((dy - dx).double()) / torch.linalg.vector_norm(dx.double())
    assert float(rel) <= U[dtype], "dx: at most a rounding apart"


def test_rms_norm_backward_against_differences(cuda_lib):
    rng = np.random.default_rng(2)
    x, w, c = rng.standard_normal((3, 24)), 1 + 0.3 * rng.standard_normal(24), rng.standard_normal((3, 24))
    loss = lambda x_, w_: float((norm_ref(x_, None, w_, 1e-3)[2] * c).sum())  # noqa: E731
    t = lambda v: torch.from_numpy(v).float().cuda()  # noqa: E731
    xd, wd, y, rstd = t(x), t(w), torch.empty(3, 24, device="cuda"), torch.empty(3, device="cuda")
    d3.rms_norm(xd, wd, y, rstd=rstd, eps=1e-3)
    dx, dw = torch.empty(3, 24, device="cuda"), torch.empty(24, device="cuda")
    d3.rms_norm_backward(t(c), xd, wd, rstd, dx, dw=dw, ws=d3.alloc_workspace(d3.rms_norm_backward_workspace_size(3, 24)))
    e = 1e-5  # central differences in float64: truncation about e^2, rounding about 1e-16 / e
    for i in range(3):
        for j in range(24):
            d = np.zeros_like(x)
            d[i, j] = e
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - float(dx[i, j])) < 1e-4
    for j in range(24):
        d = np.zeros_like(w)
        d[j] = e
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - float(dw[j])) < 1e-4


def test_no_rows(cuda_lib):
    e = lambda n: torch.empty(0, n, device="cuda")  # noqa: E731
    w, ws = torch.ones(40, device="cuda"), d3.alloc_workspace(0)
    d3.pack8(e(40), d3.alloc_packed8(0, 40))
    d3.unpack8(d3.alloc_packed8(0, 40), e(40))
    d3.rms_norm(e(40), w, e(40), rstd=torch.empty(0, device="cuda"))
    dw = torch.full((40,), 5.0, device="cuda")
    d3.rms_norm_backward(e(40), e(40), w, torch.empty(0, device="cuda"), e(40), dw=dw, accumulate=True, ws=ws)
    assert bool((dw == 5.0).all())
    d3.rms_norm_backward(e(40), e(40), w, torch.empty(0, device="cuda"), e(40), dw=dw, ws=ws)
    assert bool((dw == 0.0).all())


def test_norm_on_another_stream_and_in_a_graph(cuda_lib):
    rng = np.random.default_rng(8)
    x, w = dev(rng, 64, 2048, "bf16"), vec(rng, 2048, "bf16")
    want, y = torch.empty_like(x), torch.zeros_like(x)
    d3.rms_norm(x, w, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    d3.rms_norm(x, w, y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d3.rms_norm(x, w, y)
    g.replay()
    assert torch.equal(y, want)
