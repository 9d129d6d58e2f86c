"""The quantiser's corrected quotient (csrc/fp4.cuh, `divided`) against the rounded one, in exact arithmetic on the CPU:
a code changes only where the two lie on different sides of a tie of the grid."""
from fractions import Fraction

import numpy as np

TIES = [Fraction(1, 4), Fraction(3, 4), Fraction(5, 4), Fraction(7, 4), Fraction(5, 2), Fraction(7, 2), Fraction(5)]


def rn(v: Fraction) -> Fraction:
    """To 24 bits, ties to even (no exponent's end is near here)."""
    if v == 0:
        return v
    e = 0
    while abs(v) >= 2 ** (24 + e):
        e += 1
    while abs(v) < 2 ** (23 + e):
        e -= 1
    return Fraction(round(v / Fraction(2) ** e)) * Fraction(2) ** e


def ulp(v: Fraction) -> Fraction:
    e = 0
    while v >= Fraction(2) ** (e + 1):
        e += 1
    while v < Fraction(2) ** e:
        e -= 1
    return Fraction(2) ** (e - 23)


def corrected(x, d, r):
    q = rn(x * r)
    return rn(q + rn(x - q * d) * r)


def side(q, tie):
    return (q > tie) - (q < tie)


def test_only_one_divisor_can_change_a_code():
    """x has 8 bits (bf16), the divisor d 24, its reciprocal r is within an ulp of 1 / d (PTX: rcp.approx).  The quotient
    is near a tie only for the d around x / tie.  Among all of those, the corrected quotient is on another side than the
    rounded one for one divisor's mantissa alone, 2^24 - 1, at the tie of 1/4 and with the smaller r;
    test_gpu_v_fp4_quotient.py runs it."""
    odd = set()
    for tie in TIES:
        for m in range(128, 256):
            x = Fraction(m)
            near = rn(x / tie)
            for k in range(-6, 7):
                d = near + k * ulp(near)
                if k < 0 and d < near and ulp(d) != ulp(near):     # (below a power of two the steps are half as wide)
                    d = near + k * ulp(near) / 2
                assert rn(d) == d
                best = rn(1 / d)
                for r in (best - ulp(best) / 2, best - ulp(best), best, best + ulp(best)):
                    if rn(r) != r or abs(r - 1 / d) > ulp(1 / d):
                        continue
                    if side(corrected(x, d, r), tie) != side(rn(x / d), tie):
                        odd.add((tie, int(d / ulp(d)), r < 1 / d))
    assert odd == {(Fraction(1, 4), 2 ** 24 - 1, True)}


def test_the_block_scales_quotient_is_the_rounded_one():
    """amax / (6 g): the reciprocal is the host's rounded one.  Around every tie between E4M3 values, whatever g."""
    rng = np.random.default_rng(0)
    ties = [Fraction(2 * n + 1, 2) for n in range(8, 16)] + [Fraction(n, 2) for n in range(1, 16, 2)]
    for tie in ties:
        for m in range(128, 256):
            x = Fraction(m)
            near = rn(x / tie)
            for k in [-2, -1, 0, 1, 2, int(rng.integers(3, 1000))]:
                d = rn(near + k * ulp(near))
                r = rn(1 / d)
                assert side(corrected(x, d, r), tie) == side(rn(x / d), tie), (tie, m, k)
