"""Rotary positions in 64 bits, pair by pair, from their definition
(include/qw3.h).  Shares no code with the GPU path."""
import math

import numpy as np


def rotate(x, positions, rates, axis, style):
    """x [T, H, D], positions [A, T] (whole numbers), rates [pairs], axis [pairs] -> (rotated [T, H, D], bound).

    The bound is on what fp32 arithmetic may be off before an output is rounded.  With u and v the pair's channels:
    the angle is off by 2^-51 |t| in 64 bits (four roundings), and as a float of less than half a turn by pi 2^-24; sine
    and cosine by 2 steps of 2^-24 more; two products and a sum by 2 2^-24 (|u| + |v|): 8 2^-24 + 2^-51 |t| in all, of
    |u| + |v|."""
    x = np.asarray(x, np.float64)
    out, bound = x.copy(), np.zeros(x.shape)
    pairs = len(rates)
    for i in range(pairs):
        a, b = (i, i + pairs) if style == "halves" else (2 * i, 2 * i + 1)
        for t in range(x.shape[0]):
            angle = float(rates[i]) * int(positions[min(max(int(axis[i]), 0), len(positions) - 1)][t])
            c, s = math.cos(angle), math.sin(angle)
            u, v = x[t, :, a], x[t, :, b]
            out[t, :, a], out[t, :, b] = u * c - v * s, v * c + u * s
            bound[t, :, a] = bound[t, :, b] = (np.abs(u) + np.abs(v)) * (8 * 2.0 ** -24 + 2.0 ** -51 * abs(angle))
    return out, bound
