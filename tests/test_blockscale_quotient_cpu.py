"""The block quantiser's division-free quotient is the correctly rounded one
(CPU).

The kernels code e4m3(x / s) with s = RN(amax / 448), where RN rounds to fp32,
as q - (q s - x) r with r = RN(1 / s), q = RN(x r) and both steps fused.  For
bf16 x and amax the significands are 128 each and exponents only scale the
steps (the kernels take real divides where they could underflow), so all cases
are run through here in exact rational arithmetic.
"""
from fractions import Fraction


def rn32(v):
    """A positive or negative rational rounded to the nearest fp32 (normal
    range, ties to even)."""
    if v == 0:
        return Fraction(0)
    sign, v = (-1, -v) if v < 0 else (1, v)
    e = v.numerator.bit_length() - v.denominator.bit_length()
    if v < Fraction(2) ** e:
        e -= 1
    ulp = Fraction(2) ** (e - 23)
    n, rest = divmod(v, ulp)
    if rest * 2 > ulp or (rest * 2 == ulp and n % 2):
        n += 1
    return sign * n * ulp


def test_rn32_against_numpy():
    import numpy as np
    rng = np.random.default_rng(0)
    for v in rng.standard_normal(300) * 10.0 ** rng.integers(-20, 20, 300):
        assert float(rn32(Fraction(float(v)))) == float(np.float32(v))


def test_quotient_is_correctly_rounded_for_all_bf16_significands():
    for a in range(128, 256):
        s = rn32(Fraction(a, 128) / 448)
        r = rn32(1 / s)
        for m in range(128, 256):
            x = Fraction(m, 128)
            q = rn32(x * r)
            e = rn32(q * s - x)
            assert rn32(q - e * r) == rn32(x / s), (a, m)


def test_scale_without_a_divide_is_correctly_rounded():
    """s = RN(amax / 448) by one step on amax RN(1 / 448)."""
    r = rn32(Fraction(1, 448))
    for a in range(128, 256):
        v = Fraction(a, 128)
        q = rn32(v * r)
        e = rn32(q * 448 - v)
        assert rn32(q - e * r) == rn32(v / 448), a
