"""Plain float64 forms of the layer operators, and the error bounds the tests
hold the kernels to.  Nothing here comes from the package."""
from __future__ import annotations

import math

import numpy as np

#: Unit roundoff of the output types: 2^-p for a significand of p bits (24, 8, 11).
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
#: Half the smallest subnormal step of each type.
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
ACTS = ("none", "relu", "gelu", "silu")


def pack_ref(x):
    """Codes and scale bytes of x (float64 holding exact inputs)."""
    x = np.asarray(x, dtype=np.float64)
    t, n = x.shape
    nb = -(-n // 32)
    p = np.zeros((t, nb * 32))
    p[:, :n] = x
    p = p.reshape(t, nb, 32)
    bad = ~np.isfinite(p).all(-1)
    a = np.abs(np.where(np.isfinite(p), p, 0.0)).max(-1)
    byte = np.zeros((t, nb), dtype=np.int64)
    for i in range(t):
        for j in range(nb):
            e = -127
            if a[i, j] > 127 * 2.0 ** -127:
                e = math.frexp(a[i, j] / 127)[1]
                while a[i, j] <= 127 * 2.0 ** (e - 1):
                    e -= 1
            byte[i, j] = min(max(e, -127), 121) + 127
    with np.errstate(invalid="ignore"):
        q = np.rint(np.where(bad[..., None], 0.0, p) * 2.0 ** -(byte[..., None] - 127.0)).clip(-127, 127)
    byte[bad] = 255
    return q.reshape(t, -1)[:, :n].astype(np.int64), byte


def values_ref(codes, byte):
    """Values of codes and scale bytes, in float64."""
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return codes.astype(np.float64) * np.repeat(s, 32, axis=1)[:, :codes.shape[1]]


def act_ref(act, z):
    if act == "none":
        return z
    if act == "relu":
        return np.maximum(z, 0.0)
    u = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * sigmoid(u)


def sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1 / (1 + e), e / (1 + e))


def dact_ref(act, z):
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        s = sigmoid(z)
        return s * (1 + z * (1 - s))
    c = math.sqrt(2 / math.pi)
    th = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + th) + 0.5 * z * (1 - th ** 2) * c * (1 + 3 * 0.044715 * z ** 2)


def norm_ref(x, r, w, eps):
    h = x if r is None else x + r
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w


def norm_grad_ref(dy, h, w, rstd, dh):
    hn = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - hn * (g * hn).mean(1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * hn).sum(0)


def linear_ref(x, w, b, act, r):
    z = x @ w.T
    if b is not None:
        z = z + b
    y = act_ref(act, z)
    return z, (y if r is None else y + r)


def linear_grad_ref(dy, x, w, act, z):
    dz = dy * dact_ref(act, z) if act != "none" else dy
    return dz, dz @ w, dz.T @ x, dz.sum(0)


def sum_bound(terms: int) -> float:
    """Relative error, against the sum of magnitudes, of a sum of `terms`
    products in 32 bits, whatever the order: each of at most `terms` additions
    loses at most 2^-23 (the tensor cores may truncate) of a partial sum that
    the sum of magnitudes bounds."""
    return (terms + 4) * 2.0 ** -23


def check(got, want, tol, what):
    got, want, tol = (np.asarray(v, dtype=np.float64) for v in (got, want, tol))
    assert got.shape == want.shape, f"{what}: shape {got.shape}, want {want.shape}"
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]} against {want[bad][0]}")


def check_packed(codes, byte, want, err, what):
    """Blocks of a value known to within `err` (elementwise): each scale is the
    least that the value allows, and each code the nearest."""
    codes, byte = np.asarray(codes, dtype=np.int64), np.asarray(byte, dtype=np.int64)
    t, n = want.shape
    step = np.repeat(2.0 ** (byte - 127.0), 32, axis=1)[:, :n]
    assert (np.abs(codes) <= 127).all(), what
    check(codes * step, want, 0.5 * step + err, what)
    a = np.zeros((t, byte.shape[1] * 32))
    a[:, :n] = np.abs(want) + err
    hi = a.reshape(t, -1, 32).max(-1)
    assert ((byte == 0) | (hi > 127 * 2.0 ** (byte - 128.0))).all(), f"{what}: a scale is larger than its block needs"
