"""Float64 oracle of the cache in 4 bits (include/paged_q4.h): what a group of 16 is held as, by
enumerating the numbers that a scale and a code can be, in numpy, without any code of the library.
(The attention's oracle is oracle.paged over the values that a cache stands for.)"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

# E4M3: 4 bits of exponent (bias 7), 3 of fraction, subnormal below 2^-6, 0x7f is NaN
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest(x: Fraction, grid) -> int:
    """The place in the ascending grid of the number nearest to x >= 0; between two, the even place."""
    best = min(range(len(grid)), key=lambda i: (abs(Fraction(float(grid[i])) - x), i % 2))
    return best


def group(x):
    """(codes [16], scale code) of 16 numbers, by exact arithmetic."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(16, np.uint8), 0x7f
    top = Fraction(float(np.abs(x).max()))
    sc = max(nearest(min(top / 6, Fraction(448)), E4M3), 1)
    s = Fraction(float(E4M3[sc]))
    codes = [nearest(min(abs(Fraction(float(v))) / s, Fraction(6)), E2M1) + 8 * int(np.signbit(v)) for v in x]
    return np.array(codes, np.uint8), sc


def values(codes, scales):
    """codes [..., D / 2] bytes and scales [..., D / 16] bytes as float64 [..., D]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    m = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.append(E4M3, np.nan)[scales & 127] * np.where(scales & 128, -1.0, 1.0)
    return m * np.repeat(s, 16, -1)


def quantise(x):
    """x [..., D] as codes [..., D / 2] and scales [..., D / 16] (bytes), group by group."""
    x = np.asarray(x, np.float64)
    g = [group(v) for v in x.reshape(-1, 16)]
    codes = np.array([c for c, _ in g]).reshape(*x.shape)
    return codes[..., 0::2] | codes[..., 1::2] << 4, np.array([s for _, s in g], np.uint8).reshape(*x.shape[:-1], -1)
