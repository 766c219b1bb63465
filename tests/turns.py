"""Rotation angles to 128 bits, from integers alone."""
import numpy as np

BITS = 256
# pi to 100 digits
_PI = 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679
_PI_SCALE = 10 ** 100


def turns(f):
    """f / (2 pi) times 2^BITS, floor, for a double f (f times 2^1074 is an integer)."""
    n, d = float(f).as_integer_ratio()
    return (n * _PI_SCALE << BITS) // (2 * _PI * d)


def angles(pos, freqs):
    """Angles in radians, within half a turn of zero, of positions x frequencies: 2^-53 of each."""
    one = 1 << BITS
    t = [turns(f) for f in freqs]
    out = np.empty((len(pos), len(t)))
    for i, p in enumerate(pos):
        for j, x in enumerate(t):
            a = int(p) * x % one
            out[i, j] = (a - one if 2 * a > one else a) / one
    return out * (2 * np.pi)
