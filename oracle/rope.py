"""Rotary position embedding of one step's heads -- oracle only.

The definition, per head x of D values at position p: the first R values
form R / 2 pairs, pair i being values (i, i + R / 2), or (2i, 2i + 1) in the
interleaved form; with c, s the table's cosine and sine of angle i at p,

    a' = a c - b s,    b' = b c + a s,

and the remaining D - R values pass through.  ``rotate64`` evaluates it in
float64.  ``rotate32`` evaluates it in float32 with each product and each
sum rounded by itself (numpy rounds every operation), which is what the
library promises to the bit before the one rounding to the output type.

Only ``tests/`` may use this module.
"""

from __future__ import annotations

import numpy as np


def _rotate(x: np.ndarray, rows: np.ndarray, interleaved: bool, ft) -> np.ndarray:
    """x [N, H, D], rows [N, R] (cosines, then sines), both cast to ft."""
    x, rows = x.astype(ft), rows.astype(ft)
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half], rows[:, None, half:]
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


def rotate64(x, rows, interleaved: bool) -> np.ndarray:
    return _rotate(np.asarray(x), np.asarray(rows), interleaved, np.float64)


def rotate32(x, rows, interleaved: bool) -> np.ndarray:
    return _rotate(np.asarray(x), np.asarray(rows), interleaved, np.float32)


def angle_table(max_positions: int, rot_dim: int, base: float = 10000.0) -> np.ndarray:
    """float32 [max_positions, rot_dim] of cosines and sines of p base^(-2i/R),
    the angles in float64."""
    angle = np.arange(max_positions)[:, None] * base ** (-np.arange(0, rot_dim, 2) / rot_dim)
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
