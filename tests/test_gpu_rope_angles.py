"""Rotation tables against frequencies and angles in 60 decimal digits, at
positions where the frequencies' last bits count.

Bar: f_i / 2 pi is a whole number of 2^-64 turns to half a one and 2^-90 of
itself, so an angle is off by 2 pi 2^-64 a position at most; a value by 2^-22 of
magnitude for it (half a step of fp32, the angle's 32 bits, the two series).
"""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from tests.test_gpu_pages import P  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(d, base, scaling, factor, original, low, high):
    """Turns a position, exactly."""
    base, factor, original, low, high = (Decimal(x) for x in (base, factor, original, low, high))
    out = []
    for i in range(d // 2):
        f = (-(base.ln() * 2 * i) / d).exp()
        if scaling == "linear":
            f /= factor
        if scaling == "ntk":
            f = (-((base.ln() + factor.ln() * d / (d - 2)) * 2 * i) / d).exp()
        if scaling == "parts":
            t = min(max((original * f / (2 * PI) - low) / (high - low), Decimal(0)), Decimal(1))
            f = f * t + f / factor * (1 - t)
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("start", [0, 131072 - 4, 10 ** 9 + 7, 1 << 40])
@pytest.mark.parametrize("d,base", [(128, 10000.0), (64, 500000.0), (48, 1.0e6), (16, 1.0078125), (128, 1.0e30)])
@pytest.mark.parametrize("scaling,factor,low,high", [("plain", 1.0, 1.0, 32.0), ("linear", 3.7, 1.0, 32.0), ("ntk", 8.25, 1.0, 32.0),
                                                     ("parts", 16.0, 1.0, 32.0), ("parts", 40.0, 1.0, 4.0), ("parts", 37.5, 30.0, 31.0)])
def test_angles(P, start, d, base, scaling, factor, low, high):
    getcontext().prec = 60
    n = 9
    got = P.rope_table(n, d, base=base, scaling=scaling, factor=factor, original=8192, low_turns=low, high_turns=high,
                       magnitude=1.0, start=start).cpu().double().numpy()
    ang = np.array([[float(2 * PI * (p * t % 1)) for t in turns(d, base, scaling, factor, 8192, low, high)]
                    for p in range(start, start + n)])
    bar = 2.0 ** -22 + 2 * np.pi * 2.0 ** -64 * (start + n)
    worst = float(np.abs(got - np.concatenate([np.cos(ang), np.sin(ang)], 1)).max())
    assert worst <= bar, (worst, bar)
