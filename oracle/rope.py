"""Plain definition of rotary positions on several axes (numpy, 64 bits)."""
from __future__ import annotations

import numpy as np


def rotate(x, positions, freqs, axis, interleaved: bool, scale: float = 1.0, inverse: bool = False):
    """x [rows][heads][dim], positions [axes][rows]: the turned rows, in 64
    bits; rows that are not there (a negative position) as they were."""
    y = np.array(x, np.float64)
    half = len(freqs)
    p = np.asarray(positions, np.float64)[np.asarray(axis)] * np.asarray(freqs, np.float64)[:, None]  # [half][rows]
    p = (-p if inverse else p).T[:, None]
    c, s = scale * np.cos(p), scale * np.sin(p)
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    u, v = a * c - b * s, b * c + a * s
    out = y.copy()
    if interleaved:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = u, v
    else:
        out[..., :half], out[..., half:2 * half] = u, v
    gone = (np.asarray(positions) < 0).any(0)
    out[gone] = y[gone]
    return out


def bound(x, want, rot: int, dtype: str, scale: float = 1.0, interleaved: bool = False, turn: float = 2.0 ** -25):
    """Bound of the kernel's error: the angle is off by at most one fp32
    rounding of half a turn (pi 2^-24) and by the fixed point (position 2^-65
    turns, at most 2^-34; 2^-31 is allowed, `turn` 2^-6), sine and cosine by 2^-22, the
    three products and sum by 2^-22 of |a| + |b| together; then one rounding
    to the type (half a step, eps / 2; its subnormals)."""
    half = rot // 2
    x = np.abs(np.asarray(x, np.float64))
    both = np.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    if interleaved:
        both[..., 0:rot:2] = both[..., 1:rot:2] = a + b
    else:
        both[..., :half] = both[..., half:rot] = a + b
    fp32 = both * abs(scale) * (np.pi * 2.0 ** -24 + 2 * np.pi * turn * 2.0 ** -6 + 2.0 ** -22 + 2.0 ** -22)
    step, tiny = {"float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}[dtype]
    return fp32 + (np.abs(want) + fp32) * step + tiny
