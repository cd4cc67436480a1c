"""Float64 oracle of the 8-bit block formats and products (NumPy, no shared code with the CUDA path).

An 8-bit float is handled as the real number it stands for. e4m3: 4 mantissa
bits with the hidden one, exponents down to -6 (spacing 2^-9 below), largest
448; e5m2: 3 mantissa bits, down to -14, largest 57344.
"""
from __future__ import annotations

import numpy as np

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
_LOW = {"e4m3": -6, "e5m2": -14}
_BITS = {"e4m3": 3, "e5m2": 2}


def spacing(y, fp8: str) -> np.ndarray:
    """Distance between neighbouring values at |y|."""
    _, ex = np.frexp(np.abs(y))  # |y| = f 2^ex, f in [0.5, 1)
    return np.ldexp(1.0, np.maximum(ex - 1, _LOW[fp8]) - _BITS[fp8])


def round_nearest(y, fp8: str) -> np.ndarray:
    """The 8-bit value nearest to y, ties to even, clamped to the largest; NaN stays NaN."""
    y = np.asarray(y, np.float64)
    with np.errstate(invalid="ignore"):
        s = spacing(np.where(np.isfinite(y), y, 0.0), fp8)
        return np.clip(np.rint(y / s) * s, -TOP[fp8], TOP[fp8])


def block_scale(amax, fp8: str) -> np.ndarray:
    """2^e, e >= -126 the smallest with amax <= top 2^e; a non-finite amax is its own scale."""
    amax = np.asarray(amax, np.float64)
    ok = np.isfinite(amax)
    f, ex = np.frexp(np.where(ok, amax, 0.0) / TOP[fp8])  # division by 7 2^k: compare below, not trusting its rounding
    e = np.where(f > 0, ex, -200)
    for _ in range(2):  # at most one too high or too low
        e = np.where(np.where(ok, amax, 0.0) <= TOP[fp8] * np.ldexp(1.0, e - 1), e - 1, e)
        e = np.where(np.where(ok, amax, 0.0) > TOP[fp8] * np.ldexp(1.0, e), e + 1, e)
    return np.where(ok, np.ldexp(1.0, np.maximum(e, -126)), amax)


def _blocked(x, tile: bool):
    rows, cols = x.shape
    v = np.zeros((-(-rows // 128) * 128 if tile else rows, -(-cols // 128) * 128))
    v[:rows, :cols] = x
    return v.reshape(-1, 128, v.shape[1] // 128, 128) if tile else v.reshape(rows, -1, 128)


def quantize(x, fp8: str, tile: bool):
    """(values of the codes, scale) of a matrix; scale [cols/128, rows] by row, [rows/128, cols/128] by tile."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    v = _blocked(x, tile)
    with np.errstate(invalid="ignore", divide="ignore"):
        amax = np.abs(v).max(axis=(1, 3) if tile else 2)  # NaN propagates
        s = block_scale(amax, fp8)
        q = round_nearest(v / (s[:, None, :, None] if tile else s[:, :, None]), fp8)
    if tile:
        return q.reshape(v.shape[0] * 128, -1)[:rows, :cols], s
    return q.reshape(rows, -1)[:, :cols], s.T


def widen_rows(q, scale) -> np.ndarray:
    """The matrix a row-quantised pair stands for."""
    return np.asarray(q, np.float64) * np.repeat(np.asarray(scale, np.float64).T, 128, axis=1)[:, :q.shape[1]]


def widen_tiles(q, scale) -> np.ndarray:
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), 128, axis=0)[:q.shape[0]], 128, axis=1)[:, :q.shape[1]]
    return np.asarray(q, np.float64) * s
