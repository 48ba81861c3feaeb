"""Rotary positions and their gradient -- oracle (test infrastructure).

Not for the product path; see the package docstring.

Pair i of a band of n dimensions turns by position * f_i, f_i = base^(-2i/n),
scaled by factor s: "linear" f_i / s; "base" with base * s^(n/(n-2)); "ramp"
f_i (w + (1-w)/s), w = (c f_i / 2 pi - slow) / (fast - slow) in [0, 1] ("YaRN:
Efficient Context Window Extension of Large Language Models", section 3.2).
Positions are Python integers or int64 arrays; the angle is reduced modulo
2 pi with the integer part of the position split in 2^20 blocks, so that far
positions lose no bits to the product."""

from __future__ import annotations

import numpy as np


def frequencies(bands, base=10000.0, scaling=None, factor=1.0, context=0.0, fast=32.0, slow=1.0):
    """([pairs] radians per position in long double, [pairs] axis)."""
    f, axis = [], []
    s = np.longdouble(factor)
    two_pi = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    for a, n in enumerate(bands):
        for i in range(n // 2):
            b = np.longdouble(base)
            if scaling == "base":
                b = b * s ** (np.longdouble(n) / (n - 2))
            x = b ** (np.longdouble(-2 * i) / n)
            if scaling == "linear":
                x = x / s
            if scaling == "ramp":
                w = (np.longdouble(context) * x / two_pi - slow) / (np.longdouble(fast) - slow)
                w = min(max(w, np.longdouble(0)), np.longdouble(1))
                x = x * (w + (1 - w) / s)
            f.append(x)
            axis.append(a)
    return np.array(f, dtype=np.longdouble), np.array(axis)


def angles(pos_abl, freq, axis):
    """[B, L, pairs] angles in [0, 2 pi) of int64 positions [axes, B, L]."""
    two_pi = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    p = np.moveaxis(np.asarray(pos_abl, dtype=np.int64)[axis], 0, -1)  # [B, L, pairs]
    hi, lo = np.floor_divide(p, 1 << 20), np.mod(p, 1 << 20)
    turns = freq / two_pi
    block = np.mod(turns * (1 << 20), 1)  # turns of 2^20 positions, reduced
    t = np.mod(hi.astype(np.longdouble) * block, 1) + np.mod(lo.astype(np.longdouble) * turns, 1)
    return np.asarray(np.mod(t, 1) * two_pi, dtype=np.float64)


def rotate(x_blhd, ang, half: bool, magnitude: float = 1.0, backward: bool = False):
    """Rotated copy (float64) of [B, L, H, D] values."""
    x = np.array(x_blhd, dtype=np.float64)
    m = ang.shape[-1]
    c, s = np.cos(ang)[:, :, None] * magnitude, np.sin(ang)[:, :, None] * magnitude
    if backward:
        s = -s
    i0 = np.arange(m) if half else 2 * np.arange(m)
    i1 = i0 + (m if half else 1)
    a, b = x[..., i0].copy(), x[..., i1].copy()
    x[..., i0] = a * c - b * s
    x[..., i1] = a * s + b * c
    return x
