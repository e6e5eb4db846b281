"""A rotation's turns against exact arithmetic. No GPU."""
import ctypes
import math
from fractions import Fraction

import pytest

from test_rotary import SCALINGS, h2o  # noqa: F401


def inverse_tangent(n, bits):
    """arctan(1 / n) to `bits` bits, by its series."""
    x = power = (1 << bits + 16) // n
    for k in range(1, bits):
        power //= -n * n
        x += power // (2 * k + 1)
    return Fraction(x, 1 << bits + 16)


PI = 4 * (4 * inverse_tangent(5, 1400) - inverse_tangent(239, 1400))


def off(turns, f):
    """How far whole number `turns` is from f / (2 pi), in 2^-64 of a turn; whole turns do not count."""
    exact = Fraction(f) / (2 * PI) * 2 ** 64
    d = (turns - exact) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


def test_the_series_is_pi():
    assert abs(PI - Fraction(math.pi)) < Fraction(2) ** -52 and PI != Fraction(math.pi)
    assert f"{int(PI * 16 ** 30):x}" == "3243f6a8885a308d313198a2e037073"


@pytest.mark.parametrize("scaling,more", SCALINGS)
@pytest.mark.parametrize("dim,base", [(16, 1e4), (64, 5e5), (128, 1e4), (128, 5e5), (128, 1e6)])
def test_turns_are_rounded_once(h2o, dim, base, scaling, more):  # noqa: F811
    """Half a unit of 2^-64 of a turn, and 2^-8 more for a division by 2 pi of finitely many bits."""
    lib, f = h2o.load_library(), (ctypes.c_double * (dim // 2))()
    assert lib.h2o_rotary_frequencies(dim, base, h2o.ROTARY_SCALINGS[scaling], more.get("factor", 1.0),
                                      more.get("original", 0.0), more.get("low", 1.0), more.get("high", 32.0), f) == 0
    r = h2o.h2o_rotary(dim, base, scaling=scaling, **more)
    for i in range(dim // 2):
        assert off(r.turns[i], f[i]) <= 0.5 + 2.0 ** -8, (i, f[i])


FREQUENCIES = [1.0, 2 * math.pi * 1000.3, math.pi, 2 * math.pi, math.nextafter(2 * math.pi, 0), math.nextafter(2 * math.pi, 7),
               6 * math.pi, 0.0, 5e-324, 1e-300, 2.0 ** -64, 2.0 ** -62, 3.7e-20, 1e-3, 12345.678, 2.0 ** 31 + 0.25, 2.0 ** 40 + 1,
               1e15 + 0.125, 2.0 ** 53 - 1, 2.0 ** 53, math.nextafter(2.0 ** 53, 0), 0.1, 710 / 113]


@pytest.mark.parametrize("sign", [1, -1])
def test_given_frequencies_are_as_exact(h2o, sign):  # noqa: F811
    f = [sign * x for x in FREQUENCIES + [0.5]]
    r = h2o.h2o_rotary(2 * len(f), layout="interleaved", frequencies=f)
    for i, x in enumerate(f):
        assert off(r.turns[i], x) <= 0.5 + 2.0 ** -8, x


def test_frequencies_without_a_known_fraction_of_a_turn_are_refused(h2o):  # noqa: F811
    """Beyond 2^53 radians a position (whose neighbours are further apart than a radian)."""
    lib, r = h2o.load_library(), h2o.H2ORotary()
    for x in (math.nextafter(2.0 ** 53, math.inf), -math.nextafter(2.0 ** 53, math.inf), 1e300, -1.7e308, math.inf, math.nan):
        f = (ctypes.c_double * 8)(*[1.0] * 7, x)
        assert lib.h2o_rotary_init(ctypes.byref(r), 16, 0, f, 1.0) == -1 and b"frequencies" in lib.h2o_last_error()
