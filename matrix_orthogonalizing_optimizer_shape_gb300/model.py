"""Model operators: what stands around a stack of layers in a language model
(binding of the model part of ``include/dion3.h``).

Matrices are 2-D CUDA tensors whose rows are contiguous (any row pitch), token
numbers contiguous int32 or int64 vectors, all on the current device; outputs
are given by the caller.  Every function enqueues on ``stream`` (default: the
current one) and returns without waiting::

    d3.embedding(ids, table, x)
    d3.recurrence(z, x, h, offsets=offsets, first=state, last=state)
    d3.recurrence_backward(dh, z, x, h, dz, dx, offsets=offsets)
    d3.log_probs(logits, targets, logp, stats=stats, top_values=values, top_ids=ids)
    d3.log_probs_backward(logits, targets, stats, dlogits, dlogp=dlogp)
    d3.clip_grad_norm(grads, 1.0, norm, ws=ws)
    d3.embedding_backward(dx, ids, dtable, ws=ws)
"""
from __future__ import annotations

import array
import ctypes
import operator
import struct
from typing import Optional, Sequence

import matrix_orthogonalizing_optimizer_shape_gb300 as _d3

from . import layer as _l
from .layer import _MAT, _i32, _mat, _pm, _psz, _stream, _sz, _vec, _vp, _ws

_int, _f32 = ctypes.c_int, ctypes.c_float
SIGS = {
    "dion3_embedding": (_int, [_i32, _i32, _i32, _vp, _i32, _pm, _f32, _pm, _vp]),
    "dion3_embedding_backward_workspace_size": (_int, [_i32, _i32, _i32, _psz]),
    "dion3_embedding_backward": (_int, [_i32, _i32, _i32, _pm, _vp, _i32, _f32, _pm, _i32, _vp, _sz, _vp]),
    "dion3_recurrence": (_int, [_i32, _i32, _pm, _pm, _vp, _i32, _vp, _pm, _vp, _vp]),
    "dion3_recurrence_backward": (_int, [_i32, _i32, _pm, _pm, _pm, _pm, _vp, _i32, _vp, _vp, _pm, _pm, _vp, _vp]),
    "dion3_log_probs": (_int, [_i32, _i32, _pm, _f32, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp]),
    "dion3_log_probs_backward": (_int, [_i32, _i32, _pm, _f32, _vp, _i32, _vp, _vp, _vp, _pm, _vp]),
    "dion3_grad_norm_workspace_size": (_int, [_psz]),
    "dion3_grad_norm": (_int, [_vp, _i32, _vp, _vp, _sz, _vp]),
    "dion3_clip_grad_norm": (_int, [_vp, _vp, _i32, _f32, _vp, _vp, _sz, _vp]),
}

# dion3_tensor, as packed bytes (see the layer operators).
_TENSOR = "Pqqqi4x"
assert struct.calcsize("@" + _TENSOR) == 40
_type = operator.attrgetter("dtype")


def _ids(name: str, t, n: Optional[int], dev: int) -> tuple:
    """(data, bytes of a number) of a contiguous vector of token numbers on device `dev`."""
    if t.get_device() != dev or not t.is_cuda:
        _l._on(name, t, dev)
    if len(t.shape) != 1 or (n is not None and t.shape[0] != n) or (t.shape[0] > 1 and t.stride() != (1,)):
        raise ValueError(f"{name} must be a contiguous CUDA vector" + ("" if n is None else f" of {n}"))
    torch = _l._load_torch()
    if t.dtype is torch.int64:
        return t.data_ptr(), 8
    if t.dtype is torch.int32:
        return t.data_ptr(), 4
    raise ValueError(f"{name} must be int32 or int64, not {t.dtype}")


def embedding(ids, table, y, *, scale: float = 1.0, stream=None):
    """y[t] = scale * table[ids[t]]; zeros where ids[t] lies outside the table
    (see dion3_embedding)."""
    my = _MAT.pack(*_mat("y", y))
    (tokens, cols), dev = y.shape, y.get_device()
    mt = _MAT.pack(*_mat("table", table, None, cols, dev))
    p, b = _ids("ids", ids, tokens, dev)
    _d3._check(_l._fn("dion3_embedding")(tokens, table.shape[0], cols, p, b, mt, scale, my, _stream(stream, dev)))


def embedding_backward_workspace_size(tokens: int, vocab: int, cols: int) -> int:
    _l._sizes(tokens, vocab, cols)
    out = _sz(0)
    _d3._check(_d3.load_library().dion3_embedding_backward_workspace_size(tokens, vocab, cols, ctypes.byref(out)))
    return out.value


def embedding_backward(dy, ids, dtable, *, scale: float = 1.0, accumulate: bool = False, ws=None,
                       ws_bytes: Optional[int] = None, stream=None):
    """Gradient of :func:`embedding` for its table: dtable[v] = scale * the sum of
    dy[t] over the positions of token v, 0 where it does not occur; ``accumulate``
    adds to dtable instead (see dion3_embedding_backward)."""
    md = _MAT.pack(*_mat("dy", dy))
    (tokens, cols), dev = dy.shape, dy.get_device()
    mt = _MAT.pack(*_mat("dtable", dtable, None, cols, dev))
    p, b = _ids("ids", ids, tokens, dev)
    w, n = _ws(ws, ws_bytes, dev)
    _d3._check(_l._fn("dion3_embedding_backward")(tokens, dtable.shape[0], cols, md, p, b, scale, mt, int(accumulate),
                                                  w, n, _stream(stream, dev)))


def _offsets(t, dev: int) -> tuple:
    """(data, sequences) of the offsets of packed sequences."""
    if t is None:
        return None, 1
    p, b = _ids("offsets", t, None, dev)
    if b != 4:
        raise ValueError("offsets must be int32")
    if t.shape[0] < 1:
        raise ValueError("offsets must hold one number more than there are sequences")
    _l._sizes(t.shape[0])
    return p, t.shape[0] - 1


def _states(name: str, t, n: int, channels: int, dev: int) -> Optional[int]:
    """Address of a dense float32 [sequences, channels] tensor."""
    if t is None:
        return None
    p, ld, dtype = _mat(name, t, n, channels, dev)
    if dtype != _d3.F32 or (ld != channels and n > 1):
        raise ValueError(f"{name} must be float32 and dense")
    return p


def recurrence(z, x, h, *, offsets=None, first=None, last=None, stream=None):
    """h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(z), along the rows of each
    sequence: rows offsets[i] to offsets[i + 1], int32 (None: all rows are one).
    ``first`` and ``last`` are the states before and after each sequence, float32
    [sequences, channels].  After a state that is not finite no later one of its channel
    and sequence is (see dion3_recurrence)."""
    mz = _MAT.pack(*_mat("z", z))
    (tokens, channels), dev = z.shape, z.get_device()
    mx, mh = (_MAT.pack(*_mat(name, t, tokens, channels, dev)) for name, t in (("x", x), ("h", h)))
    p, n = _offsets(offsets, dev)
    _d3._check(_l._fn("dion3_recurrence")(tokens, channels, mz, mx, p, n, _states("first", first, n, channels, dev), mh,
                                          _states("last", last, n, channels, dev), _stream(stream, dev)))


def recurrence_backward(dh, z, x, h, dz, dx, *, offsets=None, first=None, dlast=None, dfirst=None, stream=None):
    """Gradient of :func:`recurrence` from dh and the saved z, x and h: dz, dx and
    dfirst; dlast is the gradient that reaches the states after the sequences (see
    dion3_recurrence_backward)."""
    md = _MAT.pack(*_mat("dh", dh))
    (tokens, channels), dev = dh.shape, dh.get_device()
    mz, mx, mh, mdz, mdx = (_MAT.pack(*_mat(name, t, tokens, channels, dev)) for name, t in (
        ("z", z), ("x", x), ("h", h), ("dz", dz), ("dx", dx)))
    p, n = _offsets(offsets, dev)
    _d3._check(_l._fn("dion3_recurrence_backward")(
        tokens, channels, md, mz, mx, mh, p, n, _states("first", first, n, channels, dev),
        _states("dlast", dlast, n, channels, dev), mdz, mdx, _states("dfirst", dfirst, n, channels, dev),
        _stream(stream, dev)))


def _row_values(name: str, t, rows: int, dev: int) -> Optional[int]:
    return None if t is None else _vec(name, t, rows, dev, f32=True)


def _table(name: str, t, rows: int, cols: int, dtype, dev: int) -> Optional[int]:
    """Address of a dense [rows, cols] tensor of a type."""
    if t is None:
        return None
    if not t.is_cuda or t.get_device() != dev:
        _l._on(name, t, dev)
    if t.dtype is not dtype or tuple(t.shape) != (rows, cols) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {rows} x {cols}")
    return t.data_ptr()


def log_probs(logits, targets=None, logp=None, *, scale: float = 1.0, entropy=None, stats=None, top_values=None,
              top_ids=None, stream=None):
    """Log probabilities of the targets under softmax(scale * logits) of each row,
    the entropy, and log probabilities and columns of the most probable tokens
    (float32 and int32 [rows, n], n at most 32).  ``stats``, float32 [rows, 3], is
    what :func:`log_probs_backward` needs.  Every result may be left out (see
    dion3_log_probs)."""
    ml = _MAT.pack(*_mat("logits", logits))
    (rows, vocab), dev = logits.shape, logits.get_device()
    p, b = (None, 8) if targets is None else _ids("targets", targets, rows, dev)
    top = top_values.shape[-1] if top_values is not None else top_ids.shape[-1] if top_ids is not None else 0
    torch = _l._load_torch()
    _d3._check(_l._fn("dion3_log_probs")(
        rows, vocab, ml, scale, p, b, _row_values("logp", logp, rows, dev), _row_values("entropy", entropy, rows, dev),
        _table("stats", stats, rows, 3, torch.float32, dev), top,
        _table("top_values", top_values, rows, top, torch.float32, dev),
        _table("top_ids", top_ids, rows, top, torch.int32, dev), _stream(stream, dev)))


def log_probs_backward(logits, targets, stats, dlogits, *, dlogp=None, dentropy=None, scale: float = 1.0, stream=None):
    """Gradient of :func:`log_probs` for its logits, from its stats and the gradients
    of the log probabilities and of the entropies; dlogits may be logits (see
    dion3_log_probs_backward)."""
    ml = _MAT.pack(*_mat("logits", logits))
    (rows, vocab), dev = logits.shape, logits.get_device()
    p, b = (None, 8) if targets is None else _ids("targets", targets, rows, dev)
    _d3._check(_l._fn("dion3_log_probs_backward")(
        rows, vocab, ml, scale, p, b, _table("stats", stats, rows, 3, _l._load_torch().float32, dev),
        _row_values("dlogp", dlogp, rows, dev), _row_values("dentropy", dentropy, rows, dev),
        _MAT.pack(*_mat("dlogits", dlogits, rows, vocab, dev)), _stream(stream, dev)))


def grad_norm_workspace_size() -> int:
    out = _sz(0)
    _d3._check(_d3.load_library().dion3_grad_norm_workspace_size(ctypes.byref(out)))
    return out.value


def _pack_tensors(fields: list) -> bytes:
    """dion3_tensor of each five fields (40 bytes: five 8-byte numbers)."""
    return array.array("q", fields).tobytes()


def _dense_tensors(ts: Sequence, dev: int) -> Optional[tuple]:
    """dion3_tensor of each, and their sizes, if all are dense tensors of known types on
    device `dev`.  A training step clips hundreds of tensors, whose attributes are most
    of the call: one C loop for each (50 ns a tensor; 110 through bound methods)."""
    n = len(ts)
    base = _l._load_torch()._C.TensorBase
    try:
        if dev < 0 or not all(map(base.is_contiguous, ts)) or [dev] * n != [*map(base.get_device, ts)]:
            return None
        fields = [1] * (5 * n)
        fields[4::5] = map(_l._DTYPES.__getitem__, map(_type, ts))
    except (TypeError, KeyError):  # no tensor, or no known type
        return None
    fields[0::5] = map(base.data_ptr, ts)
    fields[2::5] = fields[3::5] = sizes = [*map(base.numel, ts)]
    return _pack_tensors(fields), sizes


def _wide_mat(name: str, t, dev: int) -> tuple:
    """(data, ld, dtype) of a matrix whose sizes the call names in 64 bits."""
    shape = t.shape
    return _mat(name, t, shape[0], shape[1], dev) if len(shape) == 2 else _l._mat_checked(name, t, None, None, dev)


def _tensors(name: str, ts: Sequence, dev: int) -> bytes:
    """dion3_tensor of each: dense tensors of any shape, or matrices with contiguous rows."""
    packed = _dense_tensors(ts, dev)
    if packed is not None:
        return packed[0]
    fields = []
    for t in ts:
        if t.get_device() != dev or dev < 0:
            _l._on(name, t, dev)
        if t.is_contiguous():
            n = t.numel()
            fields += t.data_ptr(), 1, n, n, _l._dtype(t)
        else:
            p, ld, dtype = _wide_mat(name, t, dev)
            fields += p, t.shape[0], t.shape[1], ld, dtype
    return _pack_tensors(fields)


def _norm(t, dev: int) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda or t.get_device() != dev:
        _l._on("norm", t, dev)
    if t.numel() != 1 or t.dtype is not _l._load_torch().float32:
        raise ValueError("norm must be one float32")
    return t.data_ptr()


def grad_norm(tensors: Sequence, norm, *, ws=None, ws_bytes: Optional[int] = None, stream=None):
    """The norm over all elements of all tensors, of any types and shapes, into the
    one-element float32 tensor norm (see dion3_grad_norm)."""
    dev = norm.get_device()
    p = _norm(norm, dev)
    w, n = _ws(ws, ws_bytes, dev)
    _l._load_torch()
    _d3._check(_l._fn("dion3_grad_norm")(_tensors("tensors", tensors, dev), len(tensors), p, w, n, _stream(stream, dev)))


def clip_grad_norm(tensors: Sequence, max_norm: float, norm=None, *, out: Optional[Sequence] = None, ws=None,
                   ws_bytes: Optional[int] = None, stream=None):
    """Scales all tensors by min(1, max_norm / (their norm + 1e-6)), in place or into
    the tensors of ``out`` (as many elements each, in the same order, of any types);
    norm receives the norm before (see dion3_clip_grad_norm)."""
    _l._load_torch()
    dev = tensors[0].get_device() if len(tensors) else _l._device() if norm is None else norm.get_device()
    if dev < 0 and len(tensors):
        _l._on("tensors", tensors[0], dev)
    if out is not None and len(out) != len(tensors):
        raise ValueError(f"out has {len(out)} tensors, {len(tensors)} are wanted")
    if out is None:
        a, b = _tensors("tensors", tensors, dev), None
    else:
        a, b = _dense_tensors(tensors, dev), _dense_tensors(out, dev)
        if a is None or b is None or a[1] != b[1]:
            for t, o in zip(tensors, out):
                if t.shape != o.shape:
                    raise ValueError(f"out: a tensor of {tuple(o.shape)}, {tuple(t.shape)} is wanted")
            # The same rows on both sides: dense ones as rows too where the other has a pitch.
            a, b = _rows("tensors", tensors, out, dev), _rows("out", out, tensors, dev)
        else:
            a, b = a[0], b[0]
    w, n = _ws(ws, ws_bytes, dev)
    _d3._check(_l._fn("dion3_clip_grad_norm")(a, b, len(tensors), max_norm, _norm(norm, dev), w, n,
                                              _stream(stream, dev)))


def _rows(name: str, ts: Sequence, others: Sequence, dev: int) -> bytes:
    """dion3_tensor of each, by rows where it or its counterpart is not dense."""
    fields = []
    for t, o in zip(ts, others):
        if t.is_contiguous() and o.is_contiguous():
            fields.append(_tensors(name, (t,), dev))
        else:
            p, ld, dtype = _wide_mat(name, t, dev)
            fields.append(_pack_tensors([p, t.shape[0], t.shape[1], ld, dtype]))
    return b"".join(fields)
