"""Plain 64-bit restatements of the operators around a layer's products, on the
CPU, for the tests."""
import math

import numpy as np

E4M3, E2M1, E5M2, INT8, INT4, INT2 = 1, 2, 3, 4, 5, 6
EMAX = {E4M3: 8, E2M1: 2, E5M2: 15}
# (exponent of the smallest normal value, mantissa bits, largest value)
SHAPE = {E4M3: (-6, 3, 448.0), E2M1: (0, 1, 6.0), E5M2: (-14, 2, 57344.0)}


def nearest(z, fmt):
    """64-bit values to the nearest of the format, ties to even, saturated."""
    low, bits, top = SHAPE[fmt]
    e = np.maximum(np.frexp(np.abs(z))[1] - 1, low)
    step = 2.0 ** (e - bits)
    return np.clip(np.rint(z / step) * step, -top, top)


def rmsnorm(x, r, w, eps):
    """h and y in 64 bits."""
    h = x if r is None else x + r
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w


def scale_of(amax, fmt):
    """The UE8M0 code of blocks whose largest magnitude is amax (finite)."""
    e = np.frexp(amax)[1] - 1 - EMAX[fmt] + 127
    return np.where(amax == 0, 0, np.clip(e, 0, 254))


def rope(x, pos, freq, rot, factor=1.0, neighbours=False, backward=False):
    """x: tokens x heads x d in 64 bits; freq: radians a position, exact rationals
    or floats; the angle is reduced with whole numbers where freq is given in 2^-64
    turns (python ints)."""
    out = x.copy()
    for t, p in enumerate(pos):
        for i, f in enumerate(freq):
            turn = (int(p) * int(f)) % (1 << 64)
            a = 2 * math.pi * (turn / 2.0 ** 64)
            c, s = factor * math.cos(a), factor * math.sin(a) * (-1 if backward else 1)
            j, k = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
            u, v = x[t, :, j], x[t, :, k]
            out[t, :, j], out[t, :, k] = u * c - v * s, u * s + v * c
    return out
