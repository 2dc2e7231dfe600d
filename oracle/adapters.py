"""Plain definition (numpy, binary64) of the adapters of many requests and of their gradients, one
adapter at a time, with bounds on what binary32 sums and 16-bit pieces of the low-rank term may
move.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np


def rows_of(index, L):
    """The rows of each adapter, in order."""
    index = np.asarray(index, np.int64)
    return [np.flatnonzero(index == a) for a in range(L)]


def forward(base, x, index, A, B, scale):
    """(y, spread): spread bounds the error of y before its last rounding.  Per product one rounding
    of 2^-23 of the sum of magnitudes (the matrix cores may cut instead of rounding), and the
    low-rank term in two 16-bit pieces: 2^-16 of itself, or of the row's largest 2^-22."""
    M = x.shape[0]
    L, d, r = A.shape
    n = B.shape[2]
    y = np.zeros((M, d)) if base is None else base.astype(np.float64).copy()
    spread = np.zeros((M, d))
    for a, rows in enumerate(rows_of(index, L)):
        if not len(rows):
            continue
        Aa, Ba, xa, s = A[a].astype(np.float64), B[a].astype(np.float64), x[rows].astype(np.float64), float(scale[a])
        h = xa @ Ba.T
        wide = np.abs(xa) @ np.abs(Ba).T
        dh = n * 2.0 ** -23 * wide + (2.0 ** -16 + 2.0 ** -22) * np.abs(h) + 2.0 ** -22 * np.abs(h).max(1, keepdims=True)
        spread[rows] = abs(s) * (dh @ np.abs(Aa).T) + (2 * r + 4) * 2.0 ** -23 * (
            np.abs(y[rows]) + abs(s) * np.abs(h) @ np.abs(Aa).T)
        y[rows] += s * (h @ Aa.T)
    return y, spread


def backward(base, dy, x, index, A, B, scale):
    """{dx, dA, dB} and the bounds {dx, dA, dB} of their errors before the last rounding."""
    M, n = x.shape
    L, d, r = A.shape
    out = dict(dx=np.zeros((M, n)) if base is None else base.astype(np.float64).copy(), dA=np.zeros((L, d, r)),
               dB=np.zeros((L, r, n)))
    tol = {k: np.zeros_like(v) for k, v in out.items()}
    for a, rows in enumerate(rows_of(index, L)):
        if not len(rows):
            continue
        T = len(rows)
        Aa, Ba, s = A[a].astype(np.float64), B[a].astype(np.float64), float(scale[a])
        xa, ya = x[rows].astype(np.float64), dy[rows].astype(np.float64)
        h, dh = xa @ Ba.T, s * (ya @ Aa)
        hw, dhw = np.abs(xa) @ np.abs(Ba).T, abs(s) * (np.abs(ya) @ np.abs(Aa))
        # three bf16 pieces hold binary32's 24 bits, to 2^-24; binary32 sums over n, d and the rows
        out["dA"][a] = s * (ya.T @ h)
        tol["dA"][a] = (n + 6 * T + 64) * 2.0 ** -23 * abs(s) * (np.abs(ya).T @ hw)
        out["dB"][a] = dh.T @ xa
        tol["dB"][a] = (d + 6 * T + 64) * 2.0 ** -23 * (dhw.T @ np.abs(xa))
        e = d * 2.0 ** -23 * dhw + (2.0 ** -16 + 2.0 ** -22) * np.abs(dh) + 2.0 ** -22 * np.abs(dh).max(1, keepdims=True)
        tol["dx"][rows] = e @ np.abs(Ba) + (2 * r + 4) * 2.0 ** -23 * (np.abs(out["dx"][rows]) + np.abs(dh) @ np.abs(Ba))
        out["dx"][rows] += dh @ Ba
    return out, tol
