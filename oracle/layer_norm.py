"""Layer norm with weights shared by groups of rows, and its gradients --
oracle (test infrastructure).

Not for the product path; see the package docstring.

y = xhat (offset + w_g) + b_g with xhat = (x - mean) rstd, g = row //
group_rows; for dy, t = dy (offset + w_g):
dx = rstd (t - mean(t) - xhat mean(t xhat)), dw_g = sum dy xhat, db_g = sum dy."""

from __future__ import annotations

import numpy as np


def _by_row(v, rows, group_rows, missing):
    if v is None:
        return np.full((1, 1), missing)
    return np.asarray(v, np.float64)[np.arange(rows) // group_rows]


def forward(x, w, b, eps, group_rows, offset=0.0):
    """(y, mean, rstd) of x [rows, C]; w, b [groups, C] or None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    f = _by_row(w, len(x), group_rows, 1.0 - offset) + offset
    return d * rstd[:, None] * f + _by_row(b, len(x), group_rows, 0.0), mean, rstd


def backward(x, dy, w, mean, rstd, group_rows, offset=0.0):
    """(dx, dw, db) with the moments as given, and the error scales of the
    three: sums of absolute terms."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    rows, C = x.shape
    mean, rstd = (np.asarray(v, np.float64)[:, None] for v in (mean, rstd))
    u = (x - mean) * rstd
    t = dy * (_by_row(w, rows, group_rows, 1.0 - offset) + offset)
    dx = rstd * (t - t.mean(1, keepdims=True) - u * (t * u).mean(1, keepdims=True))
    a = np.abs
    sx = rstd * (a(t) + a(t).mean(1, keepdims=True) + a(u) * a(t * u).mean(1, keepdims=True))
    groups = -(-rows // group_rows)
    at = np.arange(rows) // group_rows

    def sums(v):
        out = np.zeros((groups, C))
        np.add.at(out, at, v)
        return out

    return (dx, sums(dy * u), sums(dy)), (sx, sums(a(dy * u)), sums(a(dy)))
