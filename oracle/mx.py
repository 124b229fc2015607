"""Oracle for the microscaled 4-bit formats and the layer on them (CPU, fp64).

TEST INFRASTRUCTURE ONLY -- see the package docstring.

E2M1 elements under a block scale.  MXFP4 (the Open Compute Project's
microscaling formats): blocks of 32, scale 2^e with e = floor(log2 amax) - 2,
at least -127.  NVFP4: blocks of 16, an E4M3 scale S under one scale s per row:
the smallest power of two, at least 2^-100, with amax_row <= 6 * 448 * s (1 for
a zero row); S = E4M3(amax / s / 6).  code = E2M1(x / scale); both roundings
are of the real quotient, to nearest, ties to the even code, at most 6 (448).

Everything is computed in fp64, where each step before a rounding is exact or
far finer than the distance of a quotient from a midpoint, by a search over
the listed values -- not by bit manipulation.
"""

from __future__ import annotations

import numpy as np

from .nf4 import round_bf16

MXFP4, NVFP4 = 0, 1
BLOCK = {MXFP4: 32, NVFP4: 16}

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 non-negative E4M3 values in code order (code 127 is NaN)
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119])


def nearest_even(v, values):
    """Index of the nearest of the ascending `values` to each v >= 0, ties to
    the even index, values past the last to the last."""
    mid = (values[:-1] + values[1:]) / 2
    lo = np.searchsorted(mid, v, side="left")        # number of midpoints < v
    hi = np.searchsorted(mid, v, side="right")       # number of midpoints <= v
    return np.where(hi != lo, np.where(lo % 2 == 0, lo, hi), lo)


def quantize(X, fmt: int):
    """(codes uint8 [rows, K], scale bytes [rows, K / block], row scale fp64
    [rows] or None) of a finite matrix."""
    x = np.asarray(X, dtype=np.float64)
    rows, K = x.shape
    b = BLOCK[fmt]
    s = None
    if fmt == NVFP4:
        s = np.ones(rows)
        for i, a in enumerate(np.max(np.abs(x), axis=1)):
            if a > 0:
                k = -100
                while a > 2688 * 2.0 ** k:
                    k += 1
                s[i] = 2.0 ** k
        x = x / s[:, None]
        scale = nearest_even(np.max(np.abs(x).reshape(rows, -1, b), axis=2) / 6, E4M3)
        S = E4M3[scale]
    else:
        a = np.max(np.abs(x).reshape(rows, -1, b), axis=2)
        with np.errstate(divide="ignore"):
            e = np.maximum(np.where(a > 0, np.frexp(a)[1] - 1, -1000) - 2, -127)
        scale = e + 127
        S = 2.0 ** e
    y = x.reshape(rows, -1, b)
    q = nearest_even(np.abs(y) / np.where(S == 0, 1, S)[:, :, None], E2M1)
    q = np.where(S[:, :, None] == 0, 0, q)
    codes = q + 8 * np.signbit(y)
    return codes.reshape(rows, K).astype(np.uint8), scale.astype(np.uint8), s


def scale_values(scale, fmt: int):
    scale = np.asarray(scale)
    if fmt == NVFP4:
        return np.append(E4M3, np.nan)[np.minimum(scale, 127)]
    return np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))


def dequantize(codes, scale, s, fmt: int):
    """Values in fp64."""
    codes = np.asarray(codes)
    v = E2M1[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    v = v.reshape(codes.shape[0], -1, BLOCK[fmt]) * scale_values(scale, fmt)[:, :, None]
    v = v.reshape(codes.shape)
    return v if s is None else v * np.asarray(s, dtype=np.float64)[:, None]


def pack(codes):
    """Two codes a byte, element 2j in the low nibble."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8).reshape(-1)


def unpack(packed, rows: int, cols: int):
    p = np.asarray(packed).reshape(rows, cols // 2)
    out = np.empty((rows, cols), np.uint8)
    out[:, 0::2], out[:, 1::2] = p & 15, p >> 4
    return out


def tile_scales(scale):
    """The tiled byte array of a row-major scale matrix, one byte at a time."""
    rows, cols = scale.shape
    tiles = (cols + 3) // 4
    out = np.zeros((rows + 127) // 128 * tiles * 512, np.uint8)
    for r in range(rows):
        for c in range(cols):
            out[(r // 128 * tiles + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4] = scale[r, c]
    return out


def fake_quantize(X, fmt: int):
    """deq(Q(X)) in fp64."""
    codes, scale, s = quantize(X, fmt)
    return dequantize(codes, scale, s, fmt)


def linear_fwd(X, w, A, B, alpha: float, r: int, fmt: int, Xd=None):
    """(Y, T): Y = deq(Q(X)) w^T + s (X' A^T) B^T in fp64; w the dequantised
    weight, Xd the adapter's input X' (X itself by default)."""
    Y = fake_quantize(X, fmt) @ np.asarray(w, np.float64).T
    if not r:
        return Y, None
    Xd = np.asarray(X if Xd is None else Xd, np.float64)
    T = Xd @ np.asarray(A, np.float64).T
    return Y + alpha / r * (T @ np.asarray(B, np.float64).T), T


def bf16(x):
    return round_bf16(np.asarray(x, np.float32)).astype(np.float64)
