"""Plain definition (numpy, binary64) of the gated feed-forward layer, of its backward, and of what
reads saved e4m3 codes, with bounds on what binary32 sums and functions may move.  Shares no code
with the GPU path."""
from __future__ import annotations

import math

import numpy as np

from .fplinear import e4m3_values

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def spans(offsets, T):
    return [(0, T)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def gate(g, act):
    """(act(g) / g, act'(g), bound of the relative error of the first, bound of the second's error).

    Both functions rest on one e^-w: the argument has three roundings and a constant's (4 w 2^-24
    of the result), the base-2 exponential and the reciprocal one unit each, the polynomial of
    erfc nine steps and 5e-7 < 2^-20.9: w 2^-22 + 2^-20 covers all, with w = |g| or g^2 / 2.
    The exponential and the reciprocal have no subnormal results: below 2^-126, binary32's least
    normal number, they give zero, so p carries an absolute error of up to 2^-126 as well, which
    is 2^-126 / p of it (at g = -88.5 p is 2^-127.7: e^88.5 = 2^127.7 is finite, its reciprocal 0)."""
    if act == "silu":
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-g))
            slope = p * (1.0 - p)
        w = np.abs(g)
    else:
        p = 0.5 * _erfc(-g / math.sqrt(2.0))
        slope = np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        w = 0.5 * g * g
    rel = w * 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -126 / np.maximum(p, 1e-200)
    return p, p + g * slope, rel, 3 * rel * (p + np.abs(g) * slope)


def forward(x, w, offsets, act):
    """(h, gu, h's bound, gu's bound) before the last rounding; rows in no group are NaN.
    |act'| <= 1.13 for both."""
    T, n = x.shape
    f = w.shape[1] // 2
    out = [np.full((T, k), np.nan) for k in (f, 2 * f, f, 2 * f)]
    for e, (a, b) in enumerate(spans(offsets, T)):
        if a >= b:
            continue
        gu = x[a:b] @ w[e].T
        eg = n * 2.0 ** -23 * (np.abs(x[a:b]) @ np.abs(w[e]).T)
        g, u = gu[:, :f], gu[:, f:]
        p, _, rel, _ = gate(g, act)
        h = g * p * u
        lo, hi = eg[:, :f], eg[:, f:]
        out[0][a:b], out[1][a:b], out[3][a:b] = h, gu, eg
        out[2][a:b] = (rel + 2.0 ** -22) * np.abs(h) + 1.13 * lo * (np.abs(u) + hi) + np.abs(g * p) * hi
    return out


def backward(dh, gu, act):
    """(dgu, h, dgu's bound, h's bound) of 64-bit inputs."""
    f = dh.shape[1]
    g, u = gu[:, :f], gu[:, f:]
    p, slope, rel, err = gate(g, act)
    a = g * p
    dgu = np.concatenate((dh * u * slope, dh * a), 1)
    tol = np.concatenate((np.abs(dh * u) * err, np.abs(dh * a) * rel), 1) + 2.0 ** -22 * np.abs(dgu)
    return dgu, a * u, tol, (rel + 2.0 ** -22) * np.abs(a * u)


def restore(codes, scale):
    """The numbers of codes [T, n] (uint8) and scale bytes: code x 2^(byte - 127)."""
    n = codes.shape[1]
    e = scale[:, np.arange(n) // 128].astype(np.int64) - 127
    v = np.ldexp(e4m3_values()[codes], e)
    v[scale[:, np.arange(n) // 128] == 255] = np.nan
    return v


def dw(dy, x, offsets):
    """(dW [E, d, n], bound)."""
    out, tol = [], []
    for a, b in spans(offsets, dy.shape[0]):
        b = max(a, b)
        out.append(dy[a:b].T @ x[a:b])
        tol.append((b - a) * 2.0 ** -23 * (np.abs(dy[a:b]).T @ np.abs(x[a:b])))
    return np.stack(out), np.stack(tol)
