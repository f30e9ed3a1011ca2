"""Turns of frequencies in whole numbers, apart from the library's formula: a frequency is
taken as the fraction that its double is, pi to 300 bits from Machin's formula."""
from fractions import Fraction

BITS = 300


def _atan_inverse(n):
    """atan(1 / n) * 2^BITS, cut after each term."""
    total, term, k = 0, (1 << BITS + 32) // n, 0
    while term:
        total += (-term if k & 1 else term) // (2 * k + 1)
        term //= n * n
        k += 1
    return total >> 32


PI = 4 * (4 * _atan_inverse(5) - _atan_inverse(239))        # pi * 2^BITS to a few units


def turns(radians, positions=1):
    """The angle of ``positions`` tokens at the double ``radians`` a token, in turns, modulo one:
    a Fraction in [0, 1)."""
    return Fraction(radians) * positions * (1 << BITS) / (2 * PI) % 1
