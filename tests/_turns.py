"""Fractions of a turn to as many bits as wanted, with whole numbers only."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def _pi(bits):
    """floor(pi 2^bits), by Machin's pi = 16 atan(1/5) - 4 atan(1/239)."""
    def atan(x):
        total = term = (1 << (bits + 64)) // x
        k, sign = 1, -1
        while term:
            term //= x * x
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total
    return (16 * atan(5) - 4 * atan(239)) >> 64


BITS = 400
INV_2PI = Fraction(1 << BITS, 2 * _pi(BITS))   # to about 398 bits


def turn(freq, pos=1):
    """pos * freq / (2 pi) modulo 1, in [-1/2, 1/2]."""
    x = Fraction(float(np.float32(freq))) * int(pos) * INV_2PI
    return x - round(x)


def angles(freqs, poss):
    """Angles in [-pi, pi] as float64 [len(poss)][len(freqs)]."""
    return 2 * np.pi * np.array([[float(turn(f, p)) for f in freqs] for p in poss])
