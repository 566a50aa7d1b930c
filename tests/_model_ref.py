"""Plain float64 forms of the model operators, tensors with marked surroundings,
and the error bounds the tests hold the kernels to.  Nothing here comes from the
package."""
from __future__ import annotations

import numpy as np
import torch

from _harness import torch_dtype
from _layer_ref import TINY, U, check, sum_bound  # noqa: F401

TYPES = ("f32", "bf16", "f16")


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def dev(a, dtype, pad=0, shift=0):
    """A matrix on the GPU with `pad` spare columns of NaN in its pitch, `shift`
    elements into its buffer, NaN before and behind."""
    rows, cols = a.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.from_numpy(np.asarray(a, dtype=np.float64)))
    return v


def out(rows, cols, dtype, pad=0, shift=0, fill=7.0):
    """An output filled with a marker, and its whole buffer."""
    buf = torch.full((rows * (cols + pad) + shift + 8,), fill, dtype=torch_dtype(dtype), device="cuda")
    return buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def untouched(v, buf, fill=7.0):
    """Nothing outside v's rows was written."""
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
    return bool((buf[keep] == fill).all())


def numbers(a, bits=64):
    return torch.from_numpy(np.asarray(a, dtype=np.int64)).to("cuda").to(torch.int64 if bits == 64 else torch.int32)


def embedding_ref(ids, table, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    return np.where(ok[:, None], table[np.where(ok, ids, 0)], 0.0) * scale if len(table) else np.zeros(
        (len(ids), table.shape[1]))


def embedding_grad_ref(dy, ids, vocab, scale):
    """dtable, the sums of magnitudes and the numbers of terms behind it."""
    ok = (ids >= 0) & (ids < vocab)
    d, mag, n = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1])), np.zeros(vocab)
    np.add.at(d, ids[ok], dy[ok] * scale)
    np.add.at(mag, ids[ok], np.abs(dy[ok] * scale))
    np.add.at(n, ids[ok], 1)
    return d, mag, n


def _gates(z):
    e = np.exp(-np.abs(z))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(z >= 0, big, small), np.where(z >= 0, small, big)


def recurrence_ref(z, x, offsets, first):
    """h, the states after each sequence, and a bound on the error of a state whose
    step is off by one unit: e_t = a e_{t-1} + |h_{t-1}| + |x_t|."""
    a, na = _gates(z)
    h, err = np.full_like(x, np.nan), np.zeros_like(x)
    n = len(offsets) - 1
    last = np.zeros((n, x.shape[1])) if first is None else first.copy()
    last_err = np.zeros_like(last)
    for i in range(n):
        s, e = last[i], np.zeros(x.shape[1])
        for t in range(offsets[i], offsets[i + 1]):
            e = a[t] * e + np.abs(s) + np.abs(x[t])
            s = a[t] * s + na[t] * x[t]
            h[t], err[t] = s, e
        last[i], last_err[i] = s, e
    return h, last, err, last_err


def recurrence_grad_ref(dh, z, x, h, offsets, first, dlast):
    """dz, dx, dfirst, and the same kind of bound on the error of g."""
    a, na = _gates(z)
    n = len(offsets) - 1
    dz, dx, err = np.full_like(x, np.nan), np.full_like(x, np.nan), np.zeros_like(x)
    dfirst = np.zeros((n, x.shape[1])) if dlast is None else dlast.copy()
    first_err = np.zeros_like(dfirst)
    for i in range(n):
        s, e = dfirst[i], np.zeros(x.shape[1])
        for t in range(offsets[i + 1] - 1, offsets[i] - 1, -1):
            prev = h[t - 1] if t > offsets[i] else 0.0 if first is None else first[i]
            e = e + np.abs(s) + np.abs(dh[t])
            g = dh[t] + s
            dz[t], dx[t], err[t] = g * (prev - x[t]) * a[t] * na[t], g * na[t], e
            s, e = a[t] * g, a[t] * e
        dfirst[i], first_err[i] = s, e
    return dz, dx, dfirst, err, first_err


def log_probs_ref(logits, targets, scale):
    """logp, entropy, all log probabilities; a row of -inf has log probabilities of -inf and entropy 0."""
    v = logits * scale
    m = v.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(np.isneginf(m), -np.inf, v - m)
        e = np.exp(d)
        lp = np.where(np.isneginf(m), -np.inf, d - np.log(e.sum(1, keepdims=True)))
        p = np.exp(lp)
        entropy = -np.where(p > 0, p * lp, 0.0).sum(1)
    ok = (targets >= 0) & (targets < logits.shape[1])
    logp = np.where(ok, lp[np.arange(len(lp)), np.where(ok, targets, 0)], 0.0)
    return logp, entropy + 0.0, lp


def log_probs_grad_ref(logits, targets, scale, dlogp, dentropy):
    _, entropy, lp = log_probs_ref(logits, targets, scale)
    p = np.exp(lp)
    ok = (targets >= 0) & (targets < logits.shape[1]) & ~np.isneginf(logits).all(1)
    g = np.where(ok, dlogp, 0.0)
    d = -g[:, None] * p
    d[np.arange(len(d))[ok], targets[ok]] += g[ok]
    if dentropy is not None:
        with np.errstate(invalid="ignore"):
            d -= dentropy[:, None] * np.where(p > 0, p * (lp + entropy[:, None]), 0.0)
    return d * scale


def top_ref(logits, k):
    """Columns of the k largest, equal ones in their order, NaN last."""
    v = np.where(np.isnan(logits), -np.inf, logits)
    order = np.lexsort((np.broadcast_to(np.arange(v.shape[1]), v.shape), np.isnan(logits), -v))
    return order[:, :k]
