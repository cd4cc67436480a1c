"""Float64 oracle of the AdamW step and of its 8-bit moments (NumPy, no shared code with the CUDA path)."""
from __future__ import annotations

import numpy as np

from . import fp8


def grad_norm(grads, max_norm=np.inf):
    """(norm, scale): scale = min(1, max_norm / (norm + 1e-6)), NaN when the norm is not finite in float32."""
    norm = np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads))
    with np.errstate(over="ignore"):
        finite = np.isfinite(np.float32(norm))
    return norm, min(1.0, max_norm / (norm + 1e-6)) if finite else np.nan


def step(p, g, m, v, t, *, lr, betas, eps, weight_decay, scale=1.0):
    """(p', m', v') of step t (from 1) for one tensor, every argument in float64."""
    b1, b2 = betas
    g = scale * np.asarray(g, np.float64)
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    return p - lr * weight_decay * p - lr * (m / (1.0 - b1 ** t)) / (np.sqrt(v / (1.0 - b2 ** t)) + eps), m, v


def _mix(x):
    x = (x ^ (x >> 16)) * 0x6A09E667 & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ (x >> 16)


def random16(n, seed, t, index0=0) -> np.ndarray:
    """The 16 random bits of elements index0 .. index0 + n - 1 at step t."""
    i = np.arange(index0, index0 + n, dtype=np.uint64)
    key = np.uint64(_mix((seed + t * 0x9E3779B9) & 0xFFFFFFFF))
    h = _mix((i >> np.uint64(1) & np.uint64(0xFFFFFFFF)) ^ key)
    return np.where(i & np.uint64(1), h >> np.uint64(16), h & np.uint64(0xFFFF)).astype(np.int64)


def blocks(x) -> np.ndarray:
    """Blocks of 128 consecutive elements, zeros behind the last."""
    v = np.zeros(-(-x.size // 128) * 128)
    v[:x.size] = np.asarray(x, np.float64).reshape(-1)
    return v.reshape(-1, 128)


def moment_scale(x) -> np.ndarray:
    return np.maximum(np.abs(blocks(x)).max(axis=1) / 448.0, 2.0 ** -126)


def code_steps(x, scale, u):
    """(steps, spacing): each moment's code is floor(|y| / spacing + u / 65536) spacings, y = x / scale."""
    y = blocks(x) / np.asarray(scale, np.float64)[:, None]
    s = fp8.spacing(y, "e4m3")
    return (np.abs(y) / s).reshape(-1)[:x.size] + u / 65536.0, s.reshape(-1)[:x.size]
