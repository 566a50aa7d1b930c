"""Layer operators: RMS norm, linear layer, their gradients and activations kept
in 8 bits (binding of the layer part of ``include/dion3.h``).

Arguments are 2-D CUDA tensors [tokens, features] whose rows are contiguous
(any row pitch), all on the current device; outputs are given by the caller.
Every function enqueues on ``stream`` (default: the current one) and returns
without waiting::

    x8 = d3.alloc_packed8(T, K)
    d3.rms_norm(x, gain, y, residual=r, h=h, y8=x8, rstd=rstd)
    d3.linear(y, W, out, bias=b, act=d3.ACT_SILU, z=z8)          # z8: a Packed8
    d3.linear_backward(dout, x8, W, dx=dy, dw=G, db=db, act=d3.ACT_SILU, z=z8, ws=ws)
    d3.rms_norm_backward(dy, h, gain, rstd, dx, dh=dh, dw=dgain, ws=ws)
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import matrix_orthogonalizing_optimizer_shape_gb300 as _d3

ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = range(4)

#: Columns that share one scale byte of a :class:`Packed8`.
PACK_BLOCK = 32

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class _Matrix(ctypes.Structure):
    _fields_ = [("data", _vp), ("ld", _i64), ("dtype", _i32)]


class _Packed8(ctypes.Structure):
    _fields_ = [("codes", _vp), ("ld_codes", _i64), ("scales", _vp), ("ld_scales", _i64)]


class _LinearArgs(ctypes.Structure):
    _fields_ = [("tokens", _i32), ("in_features", _i32), ("out_features", _i32), ("act", _i32),
                ("x", _Matrix), ("w", _Matrix), ("y", _Matrix), ("residual", _Matrix), ("z", _Matrix),
                ("z8", _Packed8), ("y8", _Packed8), ("bias", _vp), ("bias_dtype", _i32)]


class _LinearGradArgs(ctypes.Structure):
    _fields_ = [("tokens", _i32), ("in_features", _i32), ("out_features", _i32), ("act", _i32),
                ("accumulate", _i32),
                ("dy", _Matrix), ("w", _Matrix), ("x", _Matrix), ("z", _Matrix),
                ("x8", _Packed8), ("z8", _Packed8), ("dx", _Matrix), ("dw", _Matrix), ("db", _vp)]


_pm, _pp, _psz, _int = ctypes.POINTER(_Matrix), ctypes.POINTER(_Packed8), ctypes.POINTER(_sz), ctypes.c_int
SIGS = {
    "dion3_pack8": (_int, [_i32, _i32, _pm, _pp, _vp]),
    "dion3_unpack8": (_int, [_i32, _i32, _pp, _pm, _vp]),
    "dion3_rms_norm": (_int, [_i32, _i32, _pm, _pm, _vp, _i32, ctypes.c_float, _pm, _pm, _pp, _vp, _vp]),
    "dion3_rms_norm_backward_workspace_size": (_int, [_i32, _i32, _psz]),
    "dion3_rms_norm_backward": (_int, [_i32, _i32, _pm, _pm, _vp, _i32, _vp, _pm, _pm, _vp, _i32, _vp, _sz, _vp]),
    "dion3_linear_workspace_size": (_int, [_i32, _i32, _i32, _i32, _i32, _psz]),
    "dion3_linear": (_int, [ctypes.POINTER(_LinearArgs), _vp, _sz, _vp]),
    "dion3_linear_backward_workspace_size": (_int, [_i32, _i32, _i32, _i32, _i32, _psz]),
    "dion3_linear_backward": (_int, [ctypes.POINTER(_LinearGradArgs), _vp, _sz, _vp]),
}

# A call is marshalled as packed bytes in the layout of the structures above: a
# small operator's time is its host side, and filling ctypes structures field by
# field took longer than the rest of the call.
_MAT = struct.Struct("@Pqi4x")
_PACK = struct.Struct("@PqPq")
_LINEAR = struct.Struct("@4i" + "Pqi4x" * 5 + "PqPq" * 2 + "Pi4x")
_LINEAR_GRAD = struct.Struct("@5i4x" + "Pqi4x" * 4 + "PqPq" * 2 + "Pqi4x" * 2 + "P")
assert (_MAT.size, _PACK.size, _LINEAR.size, _LINEAR_GRAD.size) == tuple(
    map(ctypes.sizeof, (_Matrix, _Packed8, _LinearArgs, _LinearGradArgs)))
_NO_MAT, _NO_PACK = (0, 0, 0), (0, 0, 0, 0)

#: The largest size that a call can name: ctypes keeps the low 32 bits of a larger one.
_MOST = 2 ** 31 - 1


def _sizes(*sizes: int):
    """Refuses sizes that a call cannot name."""
    if max(sizes) > _MOST:
        raise ValueError(f"a size of {max(sizes)} is larger than any operator takes")


_FNS = {}
_torch = _I8 = _U8 = None
_DTYPES = {}


def _load_torch():
    """torch, and the dtypes' codes (on first use: importing this module needs neither)."""
    global _torch, _I8, _U8
    if _torch is None:
        import torch
        _I8, _U8 = torch.int8, torch.uint8
        _DTYPES.update({torch.float32: _d3.F32, torch.bfloat16: _d3.BF16, torch.float16: _d3.F16})
        _torch = torch
    return _torch


def _fn(name: str):
    """The library's entry point, taking structures as bytes."""
    f = _FNS.get(name)
    if f is None:
        _load_torch()
        res, args = _d3._SIGS[name]
        args = [_vp if isinstance(a, type) and issubclass(a, ctypes._Pointer) else a for a in args]
        f = _FNS[name] = ctypes.CFUNCTYPE(res, *args)((name, _d3.load_library()))
    return f


def _dtype(t) -> int:
    """dion3_dtype of a tensor."""
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        pass
    _load_torch()
    if t.dtype not in _DTYPES:
        raise ValueError(f"dtype {t.dtype} is not float32, bfloat16 or float16")
    return _DTYPES[t.dtype]


def _device() -> int:
    """The current device, where the kernels run."""
    return (_torch or _load_torch())._C._cuda_getDevice()


def _stream(stream, dev: int) -> Optional[int]:
    """The stream of a call whose tensors are on device `dev`."""
    current = _device()
    if dev != current:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{current}")
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(current) or None
    return _d3._stream(stream)


def _on(name: str, t, dev: Optional[int]):
    """Refuses a tensor that is not on device `dev` (None: any CUDA device)."""
    if not t.is_cuda:
        raise ValueError(f"{name} is not a CUDA tensor")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's other tensors are on device cuda:{dev}")


def _mat(name: str, t, rows: Optional[int] = None, cols: Optional[int] = None, dev: Optional[int] = None) -> tuple:
    """(data, ld, dtype) of a 2-D CUDA tensor with contiguous rows; shape and device checked where given."""
    try:
        (r, c), (ld, inner) = t.shape, t.stride()
        if ((t.is_cuda if dev is None else t.get_device() == dev) and inner == 1 and ld >= c
                and (r <= _MOST if rows is None else r == rows) and (c <= _MOST if cols is None else c == cols)):
            return t.data_ptr(), ld, _DTYPES[t.dtype]
    except (ValueError, KeyError):
        pass
    return _mat_checked(name, t, rows, cols, dev)


def _mat_checked(name: str, t, rows, cols, dev) -> tuple:
    """The same, case by case: what is wrong, or the layouts whose strides say nothing."""
    _on(name, t, dev)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} has {len(shape)} dimensions, 2 are wanted")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} is {r} x {c}, {rows if rows is not None else r} x "
                         f"{cols if cols is not None else c} is wanted")
    _sizes(r if rows is None else 0, c if cols is None else 0)
    ld, inner = t.stride()
    if inner != 1 and c > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if ld < c:  # one row (any stride), or rows that overlap
        if r > 1:
            raise ValueError(f"{name}: rows overlap")
        ld = c
    return t.data_ptr(), ld, _dtype(t)


def _vec(name: str, t, n: int, dev: Optional[int] = None, f32: bool = False) -> int:
    if not t.is_cuda if dev is None else t.get_device() != dev:
        _on(name, t, dev)
    if t.shape != (n,) or (n > 1 and t.stride() != (1,)):
        raise ValueError(f"{name} must be a contiguous CUDA vector of {n}")
    if f32 and _dtype(t) != _d3.F32:
        raise ValueError(f"{name} must be float32")
    return t.data_ptr()


class Packed8:
    """A matrix in 8-bit blocks (``dion3_packed8``): int8 codes [rows, cols] and
    uint8 scale bytes [rows, ceil(cols / 32)], rows contiguous, any row pitch
    (multiples of 16 bytes are fastest, see :func:`alloc_packed8`).  A call reads
    the addresses that ``codes`` and ``scales`` have when it is made, so both may
    be replaced (moved to the host and back, for instance)."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes, scales):
        self.codes, self.scales = codes, scales
        _packed("Packed8", self)

    @property
    def shape(self):
        return tuple(self.codes.shape)


def _packed(name: str, p: Packed8, rows: Optional[int] = None, cols: Optional[int] = None,
            dev: Optional[int] = None) -> tuple:
    """(codes, ld_codes, scales, ld_scales); shape and device checked where given."""
    q, s = p.codes, p.scales
    try:
        (r, c), (sr, nb), (lq, qi), (ls, si), d = q.shape, s.shape, q.stride(), s.stride(), q.get_device()
        if (qi == 1 and si == 1 and lq >= c and ls >= nb and sr == r and nb == (c + 31) // 32
                and (rows is None or (r == rows and c == cols)) and q.dtype is _I8 and s.dtype is _U8
                and d >= 0 and s.get_device() == d and (dev is None or d == dev)):
            return q.data_ptr(), lq, s.data_ptr(), ls
    except ValueError:
        pass
    return _packed_checked(name, q, s, rows, cols, dev)


def _packed_checked(name: str, q, s, rows, cols, dev) -> tuple:
    """The same, case by case (see _mat_checked)."""
    t = _load_torch()
    if q.dtype != t.int8 or s.dtype != t.uint8:
        raise ValueError(f"{name}: codes must be int8 and scales uint8")
    if not (q.is_cuda and s.is_cuda) or q.dim() != 2 or s.dim() != 2:
        raise ValueError(f"{name}: codes and scales must be 2-D CUDA tensors")
    _on(f"{name}: codes", q, s.get_device() if dev is None else dev)
    _on(f"{name}: scales", s, q.get_device())
    r, c = q.shape
    if rows is not None and (r, c) != (rows, cols):
        raise ValueError(f"{name} is {r} x {c}, {rows} x {cols} is wanted")
    nb = -(-c // PACK_BLOCK)
    if tuple(s.shape) != (r, nb):
        raise ValueError(f"{name}: scales must be {r} x {nb} for codes of {r} x {c}")
    lds = []
    for m, n in ((q, c), (s, nb)):
        ld, inner = m.stride()
        if (inner != 1 and n > 1) or (ld < n and r > 1):
            raise ValueError(f"{name}: the rows of codes and scales must be contiguous and not overlap")
        lds.append(max(ld, n))
    return q.data_ptr(), lds[0], s.data_ptr(), lds[1]


def alloc_packed8(rows: int, cols: int, device=None) -> Packed8:
    """An uninitialised :class:`Packed8` with row pitches that are multiples of 16 bytes."""
    import torch
    dev = device if device is not None else "cuda"
    nb = -(-cols // PACK_BLOCK)
    codes = torch.empty(rows, -(-cols // 16) * 16, dtype=torch.int8, device=dev)[:, :cols]
    scales = torch.empty(rows, -(-nb // 16) * 16, dtype=torch.uint8, device=dev)[:, :nb]
    return Packed8(codes, scales)


def _ws(ws, nbytes, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev:
        _on("ws", ws, dev)
    return ws.data_ptr(), nbytes if nbytes is not None else ws.numel() * ws.element_size()


def pack8(x, out: Packed8, stream=None):
    """x [rows, cols] into 8-bit blocks (see dion3_pack8)."""
    m = _MAT.pack(*_mat("x", x))
    (rows, cols), dev = x.shape, x.get_device()
    _d3._check(_fn("dion3_pack8")(rows, cols, m, _PACK.pack(*_packed("out", out, rows, cols, dev)),
                                  _stream(stream, dev)))


def unpack8(src: Packed8, out, stream=None):
    """The values that 8-bit blocks stand for, in out's dtype (see dion3_unpack8)."""
    p = _PACK.pack(*_packed("src", src))
    (rows, cols), dev = src.codes.shape, src.codes.get_device()
    _sizes(rows, cols)
    _d3._check(_fn("dion3_unpack8")(rows, cols, p, _MAT.pack(*_mat("out", out, rows, cols, dev)),
                                    _stream(stream, dev)))


def _opt(name: str, t, rows: int, cols: int, dev: int):
    return None if t is None else _MAT.pack(*_mat(name, t, rows, cols, dev))


def rms_norm(x, weight, y=None, *, residual=None, h=None, y8: Optional[Packed8] = None, rstd=None,
             eps: float = 1e-6, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over each row, y
    and / or its 8-bit blocks y8, and rstd for the backward pass (see
    dion3_rms_norm)."""
    mx = _MAT.pack(*_mat("x", x))
    (rows, cols), dev = x.shape, x.get_device()
    _d3._check(_fn("dion3_rms_norm")(
        rows, cols, mx, _opt("residual", residual, rows, cols, dev), _vec("weight", weight, cols, dev), _dtype(weight),
        eps, _opt("h", h, rows, cols, dev), _opt("y", y, rows, cols, dev),
        None if y8 is None else _PACK.pack(*_packed("y8", y8, rows, cols, dev)),
        None if rstd is None else _vec("rstd", rstd, rows, dev, f32=True), _stream(stream, dev)))


def rms_norm_backward_workspace_size(rows: int, cols: int) -> int:
    _sizes(rows, cols)
    out = _sz(0)
    _d3._check(_d3.load_library().dion3_rms_norm_backward_workspace_size(rows, cols, ctypes.byref(out)))
    return out.value


def rms_norm_backward(dy, h, weight, rstd, dx, *, dh=None, dw=None, accumulate: bool = False, ws=None,
                      ws_bytes: Optional[int] = None, stream=None):
    """Gradient of :func:`rms_norm`: dx (of x and the residual alike; dh is the
    gradient that reaches h from elsewhere) and dw, float32 (see
    dion3_rms_norm_backward)."""
    mdy = _MAT.pack(*_mat("dy", dy))
    (rows, cols), dev = dy.shape, dy.get_device()
    p, n = _ws(ws, ws_bytes, dev)
    _d3._check(_fn("dion3_rms_norm_backward")(
        rows, cols, mdy, _opt("h", h, rows, cols, dev), _vec("weight", weight, cols, dev), _dtype(weight),
        _vec("rstd", rstd, rows, dev, f32=True), _opt("dh", dh, rows, cols, dev), _opt("dx", dx, rows, cols, dev),
        None if dw is None else _vec("dw", dw, cols, dev, f32=True), int(accumulate), p, n, _stream(stream, dev)))


def _ws_size(fn: str, tokens, in_features, out_features, dtype, strided) -> int:
    import torch
    code = {torch.float32: _d3.F32, torch.bfloat16: _d3.BF16, torch.float16: _d3.F16}.get(dtype, -1)
    _sizes(tokens, in_features, out_features)
    out = _sz(0)
    _d3._check(getattr(_d3.load_library(), fn)(tokens, in_features, out_features, code, int(strided),
                                               ctypes.byref(out)))
    return out.value


def linear_workspace_size(tokens: int, in_features: int, out_features: int, *, dtype, strided: bool = False) -> int:
    """Workspace bytes of :func:`linear` (0 for dense tensors with in_features a
    multiple of 64; needed only where it is no multiple of 8, and else a help to
    large products); ``strided``: for any pitch and base."""
    return _ws_size("dion3_linear_workspace_size", tokens, in_features, out_features, dtype, strided)


def linear_backward_workspace_size(tokens: int, in_features: int, out_features: int, *, dtype,
                                   strided: bool = False) -> int:
    """Workspace bytes of :func:`linear_backward`; ``strided``: for any pitch and base."""
    return _ws_size("dion3_linear_backward_workspace_size", tokens, in_features, out_features, dtype, strided)


def linear(x, w, y, *, bias=None, residual=None, act: int = ACT_NONE, z=None, y8: Optional[Packed8] = None, ws=None,
           ws_bytes: Optional[int] = None, stream=None):
    """y = act(x w^T + bias) + residual.  z (a tensor or a :class:`Packed8`)
    receives the pre-activation, y8 the output in 8-bit blocks (see
    dion3_linear)."""
    mx = _mat("x", x)
    (tokens, k), dev = x.shape, x.get_device()
    mw = _mat("w", w, None, k, dev)
    n = w.shape[0]
    z8 = _NO_PACK
    mz = _NO_MAT
    if isinstance(z, Packed8):
        z8 = _packed("z", z, tokens, n, dev)
    elif z is not None:
        mz = _mat("z", z, tokens, n, dev)
    args = _LINEAR.pack(tokens, k, n, act, *mx, *mw, *_mat("y", y, tokens, n, dev),
                        *(_NO_MAT if residual is None else _mat("residual", residual, tokens, n, dev)), *mz, *z8,
                        *(_NO_PACK if y8 is None else _packed("y8", y8, tokens, n, dev)),
                        0 if bias is None else _vec("bias", bias, n, dev), 0 if bias is None else _dtype(bias))
    p, nb = _ws(ws, ws_bytes, dev)
    _d3._check(_fn("dion3_linear")(args, p, nb, _stream(stream, dev)))


def linear_backward(dy, x, w, *, dx=None, dw=None, db=None, act: int = ACT_NONE, z=None, accumulate: bool = False,
                    ws=None, ws_bytes: Optional[int] = None, stream=None):
    """Gradient of :func:`linear` from dy: dx, dw (any dtype) and db (float32),
    those that are given.  x and z are tensors or
    :class:`Packed8` checkpoints; ``accumulate`` adds to dw and db (see
    dion3_linear_backward)."""
    mdy = _mat("dy", dy)
    (tokens, n), dev = dy.shape, dy.get_device()
    mw = _mat("w", w, n, None, dev)
    k = w.shape[1]
    mx, x8, mz, z8 = _NO_MAT, _NO_PACK, _NO_MAT, _NO_PACK
    if isinstance(x, Packed8):
        x8 = _packed("x", x, tokens, k, dev)
    elif x is not None:
        mx = _mat("x", x, tokens, k, dev)
    if isinstance(z, Packed8):
        z8 = _packed("z", z, tokens, n, dev)
    elif z is not None:
        mz = _mat("z", z, tokens, n, dev)
    args = _LINEAR_GRAD.pack(tokens, k, n, act, int(accumulate), *mdy, *mw, *mx, *mz, *x8, *z8,
                             *(_NO_MAT if dx is None else _mat("dx", dx, tokens, k, dev)),
                             *(_NO_MAT if dw is None else _mat("dw", dw, n, k, dev)),
                             0 if db is None else _vec("db", db, n, dev, f32=True))
    p, nb = _ws(ws, ws_bytes, dev)
    _d3._check(_fn("dion3_linear_backward")(args, p, nb, _stream(stream, dev)))
