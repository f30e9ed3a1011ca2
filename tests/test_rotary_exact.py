"""Frequencies of rotations against exact ones: what a rotation stores is the double that it
was given, in units of 2^-64 of a turn modulo one turn, to half a unit."""
import math
import random
from decimal import Decimal, localcontext
from fractions import Fraction

import pytest

import rotary_exact as exact
from paged_kv_cache_255_gb300 import pagedattn as pa

UNIT = Fraction(1, 1 << 64)


def apart(turn, want):
    d = abs(Fraction(int(turn), 1 << 64) - want)
    return min(d, 1 - d)


def test_pi():
    assert abs(Fraction(exact.PI, 1 << exact.BITS) - Fraction(math.pi)) < Fraction(1, 1 << 52)
    assert str(exact.PI * 10 ** 40 >> exact.BITS) == "31415926535897932384626433832795028841971"


def test_given_frequencies_are_exact(pa_lib):
    rng = random.Random(4)
    f = [0.0, -0.0, 1.0, -1.0, math.pi, 2 * math.pi, -2 * math.pi, 2.0 ** 20, -(2.0 ** 20), math.nextafter(2.0 ** 20, 0.0),
         1000.125, 6.5, 1e-12, 2.0 ** -30, 2.0 ** -61, 2.0 ** -62, -(2.0 ** -63), 5e-324, -1e-300, 1e-30]
    f += [rng.choice([-1, 1]) * 2.0 ** rng.uniform(-70, 20) for _ in range(1004)]
    for i in range(0, len(f), 64):
        R = pa.Rotary(128, frequencies=f[i:i + 64])
        for t, x in zip(R._struct.turns, f[i:i + 64]):
            assert apart(t, exact.turns(x)) <= UNIT * Fraction(51, 100), (x, t)


@pytest.mark.parametrize("rot_dim,base", [(128, 10000.0), (64, 500000.0), (16, 1.5), (96, 1e6)])
def test_powers_of_the_base(pa_lib, rot_dim, base):
    R = pa.Rotary(rot_dim, base=base)
    with localcontext() as c:
        c.prec = 60
        for i, t in enumerate(R._struct.turns[:rot_dim // 2]):
            # the exponent and the power as doubles: their roundings, the former's times ln(base)
            theta = Fraction(Decimal(base) ** (Decimal(-2 * i) / Decimal(rot_dim)))
            rel = Fraction(2 + math.log(base)) * Fraction(1, 1 << 53)
            want = theta * (1 << exact.BITS) / (2 * exact.PI)
            assert apart(t, want % 1) <= want * rel + UNIT
