"""Angles of the position rotation in whole numbers, from pi and the frequency's own value: an oracle that shares no
arithmetic with the binding. Test infrastructure."""
import math
from fractions import Fraction

PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def fraction(f: float) -> Fraction:
    """Turns a position of a frequency of f radians."""
    return Fraction(f) / (2 * PI)


def slack(f: float) -> Fraction:
    """How far the binding's fraction may be off: it divides by the double next to 2 pi (0.36 of 2^-53 under it), rounds the
    quotient (2^-53 at most) and the product with 2^64 to a whole number (half of one)."""
    return abs(fraction(f)) * Fraction(137, 100) / 2 ** 53 + Fraction(1, 2 ** 65)


def angle(f: float, position: int) -> float:
    """Radians in [0, 2 pi)."""
    t = fraction(f) * position
    return float(t - math.floor(t)) * 2 * math.pi
