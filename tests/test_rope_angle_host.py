"""How far off an angle of qk_norm_rope may be, on the host: its float64 steps in exact arithmetic (CPU only).

turn = position * (inv_freq * (1 / 2 pi)), each product rounded once and the constant once: less than 3 * 2^-53 (1 + 2^-52) of the
angle, so below 2^-51 of it.  Taking off whole turns and doubling are exact, and rounding the rest, at most half a turn, to
float32 moves it by at most 2^-25 of half a turn, 2^-23 of a radian."""
import random
import struct
from fractions import Fraction

PI = Fraction(31415926535897932384626433832795028841971693993751058209749, 10 ** 58)       # to 58 places


def f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


def off(position, freq):
    """Radians between the angle that is rotated by and position * freq, and the angle; the first part without the last rounding."""
    turn = float(position) * (freq * 0.15915494309189535)
    rest = Fraction(turn) - round(turn)
    last = f32(float(2 * rest))
    want = Fraction(position) * Fraction(freq)
    return float(abs(Fraction(turn) * 2 * PI - want)), float(abs(Fraction(last) - 2 * rest) * PI), float(abs(want))


def test_angles():
    r = random.Random(1)
    cases = [(1349035241, f32(1.5873595)), (2 ** 31 - 1, 1.0), (-2 ** 31, f32(0.999999)), (5, f32(1e-7)), (0, 1.0), (1, f32(3.4e38))]
    cases += [(r.randint(-2 ** 31, 2 ** 31 - 1), f32(2.0 ** r.uniform(-30, 8))) for _ in range(20000)]
    for position, freq in cases:
        first, last, angle = off(position, freq)
        assert first <= 2.0 ** -51 * angle and last <= 2.0 ** -23, (position, freq)


def test_the_angle_counts():
    # below 2^31 the steps in float64 alone can pass 2^-21: the bound is not one of the last steps' alone
    first, _, angle = off(1349035241, f32(1.5873595))
    assert angle < 2 ** 31 and first > 2.0 ** -21
