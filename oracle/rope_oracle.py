"""Plain CPU oracle for the rotation of heads by position (numpy, float64; TEST
INFRASTRUCTURE ONLY, no code shared with the CUDA path).

Pair j of a head turns by angle = position[axis of j] * inv_freq[j]; its elements are
j and j + pairs, or 2 j and 2 j + 1 where pairs lie side by side:
    (x, y) -> (x cos - y sin, x sin + y cos).
The angle is reduced to a turn in exact integers, so that its error is that of pi's
60 digits and of one float64, whatever the position.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


def angle(position: int, frequency: float) -> float:
    """position * frequency modulo 2 pi, in (-pi, pi]."""
    turns = Fraction(frequency) * int(position) / TWO_PI
    return float((turns - round(turns)) * TWO_PI)


def rope(x, inv_freq, positions, pair_axis=None, interleaved=False, inverse=False):
    """x [B, n, heads, dim] (float64) turned; positions [axes, B, n] integers.  Also the
    largest |x| + |y| of each element's pair, which bounds what an angle's error does."""
    x = np.asarray(x, dtype=np.float64)
    out, size = x.copy(), np.abs(x)
    B, n = x.shape[:2]
    pairs = len(inv_freq)
    for j in range(pairs):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
        axis = 0 if pair_axis is None else int(pair_axis[j])
        for s in range(B):
            for i in range(n):
                t = angle(int(positions[axis][s][i]), float(inv_freq[j])) * (-1.0 if inverse else 1.0)
                c, w = math.cos(t), math.sin(t)
                u, v = x[s, i, :, a], x[s, i, :, b]
                out[s, i, :, a], out[s, i, :, b] = u * c - v * w, u * w + v * c
                size[s, i, :, a] = size[s, i, :, b] = np.abs(u) + np.abs(v)
    return out, size
