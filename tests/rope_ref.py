"""Rotary positions and FP8 rows in 64 bits, for the tests: angles reduced as exact
fractions, so that the reference holds at every int32 position."""
import math
from fractions import Fraction

import torch

# 2 pi to 50 digits
TWO_PI = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)


def angles(positions, inv_freq, axis_of_pair):
    """positions [axes][n] ints -> (cos, sin) float64 [n, pairs]."""
    n = len(positions[0])
    inv = [Fraction(f) for f in inv_freq]
    cos, sin = [], []
    for i in range(n):
        t = [positions[a][i] * f for a, f in zip(axis_of_pair, inv)]
        t = [float(x - TWO_PI * math.floor(x / TWO_PI)) for x in t]
        cos.append([math.cos(x) for x in t])
        sin.append([math.sin(x) for x in t])
    return torch.tensor(cos, dtype=torch.float64), torch.tensor(sin, dtype=torch.float64)


def turn(x, cos, sin, rot, interleaved, scale=1.0):
    """x [n, heads, d] -> (turned float64, |x_a| + |x_b| of each value's pair)."""
    x = x.double().cpu()
    y, mag = x.clone(), x.abs()
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    c, s = cos[:, None], sin[:, None]
    y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
    y[..., b] = scale * (x[..., b] * c + x[..., a] * s)
    both = abs(scale) * (x[..., a].abs() + x[..., b].abs())
    mag[..., a], mag[..., b] = both, both
    return y, mag


# The kernel's angle is off by at most 2 pi 2^-32 (the fraction of a turn) + pi 2^-24 (its
# conversion to fp32), its cos and sin by two fp32 units more, and two products and a sum
# round three times: below 2^-20 of |x_a| + |x_b| in all.  Then bf16, half a step: 2^-8.
FP32_PART = 2.0 ** -20


def bf16_limit(ref, mag):
    return (ref.abs() + FP32_PART * mag) * 2.0 ** -8 + FP32_PART * mag
