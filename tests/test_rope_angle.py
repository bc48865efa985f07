"""The accuracy that csrc/rope.cuh states for the reduced angle: the same doubles against exact rationals."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import serving

# 1 / (2 pi) from 60 digits of pi
INV_2PI = 1 / (2 * Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59))


@pytest.mark.parametrize("bits,bound", [(17, 2.0 ** -37), (24, 2.0 ** -30), (31, 2.0 ** -23)])
def test_reduced_angle(bits, bound):
    rng = np.random.default_rng(bits)
    freqs = np.concatenate([serving.rope_freqs(64)[:12], serving.rope_freqs(128, base=500000.0)[:12]])
    pos = np.concatenate([2 ** bits - 1 - np.arange(40), rng.integers(2 ** (bits - 1), 2 ** bits, 200)])
    worst = 0.0
    for f in freqs:
        turns = pos.astype(np.float64) * (f * 0.15915494309189533576888)
        left = turns - np.rint(turns)
        for p, r in zip(pos.tolist(), left.tolist()):
            exact = p * Fraction(float(f)) * INV_2PI
            off = Fraction(r) - exact
            worst = max(worst, abs(float(off - round(off))))
    assert worst <= bound, f"{worst:.3e}"
    assert worst >= bound / 16, "the bound is idle"
