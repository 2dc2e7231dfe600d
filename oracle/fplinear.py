"""Plain definitions (numpy, binary64) of the floating-point linear layers and of gradient
clipping.  They share no code with the GPU path: codes come from a table of all e4m3 values,
products from binary64 matrix products one group at a time, sums from math.fsum."""
from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 OCP e4m3 codes (0x7F and 0xFF are NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v[c] = math.nan if c & 0x7F == 0x7F else (-x if c & 0x80 else x)
    return v


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:0x7F]  # ascending, code = index


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values, half to even; |x| <= 464 (which rounds to 448)."""
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 0x7E)
    lo = hi - 1
    down, up = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def scale_exponent(a: float) -> int:
    """The least e >= -127 with a 2^-e <= 448; 0 for a = 0."""
    if a == 0:
        return 0
    e = -160
    while math.ldexp(a, -e) > 448.0:
        e += 1
    return max(e, -127)


def quantize(x: np.ndarray, rows: int):
    """(codes, scale bytes [R', 4 ceil(C / 512)]) of x [R, C] in blocks of rows x 128."""
    R, C = x.shape
    codes = np.empty((R, C), np.uint8)
    scale = np.full((-(-R // rows), 4 * -(-C // 512)), 127, np.uint8)
    for i in range(0, R, rows):
        for j in range(0, C, 128):
            b = x[i:i + rows, j:j + 128].astype(np.float64)
            if not np.isfinite(b).all():
                scale[i // rows, j // 128] = 255
                codes[i:i + rows, j:j + 128] = 0x7F
                continue
            e = scale_exponent(float(np.abs(b).max()))
            scale[i // rows, j // 128] = e + 127
            codes[i:i + rows, j:j + 128] = to_e4m3(np.ldexp(b, -e))
    return codes, scale


def dequantize(codes: np.ndarray, scale: np.ndarray, rows: int) -> np.ndarray:
    R, C = codes.shape
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    s = np.repeat(np.repeat(s, rows, 0)[:R], 128, 1)[:, :C]
    return _VALUES[codes] * s


def boundaries(offsets, M: int) -> list[int]:
    """Row boundaries of the groups: each offset forced into [0, M] and above its predecessors."""
    out, top = [], 0
    for o in offsets:
        top = max(top, min(max(int(o), 0), M))
        out.append(top)
    return out


def grouped(x, offsets, w):
    """(Y, the sum of |x| |w| behind each output) of x [M, n], w [E, d, n]; NaN in rows of no group."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = np.zeros_like(y)
    b = boundaries(offsets, x.shape[0])
    for e in range(len(b) - 1):
        r = slice(b[e], b[e + 1])
        y[r] = x[r] @ w[e].T
        mag[r] = np.abs(x[r]) @ np.abs(w[e]).T
    return y, mag


def grouped_dw(dy, x, offsets):
    """(dW [E, d, n], the sum of |dy| |x| behind each entry, rows of each group)."""
    b = boundaries(offsets, x.shape[0])
    E = len(b) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(dw)
    for e in range(E):
        r = slice(b[e], b[e + 1])
        dw[e] = dy[r].T @ x[r]
        mag[e] = np.abs(dy[r]).T @ np.abs(x[r])
    return dw, mag, np.diff(b)


def sumsq(grads) -> float:
    return math.fsum(math.fsum((g.astype(np.float64) ** 2).ravel().tolist()) for g in grads)


def clip_factor(total: float, max_norm: float) -> float:
    return min(1.0, max_norm / (math.sqrt(total) + 1e-6))
