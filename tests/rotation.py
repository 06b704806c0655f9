"""Plain form of the position rotation (numpy): angles in extended precision, products in fp64."""
import numpy as np


def factors(pos, freqs, amplitude):
    """amplitude * (cos, sin) of pos * freqs: [..., rot / 2].  The 64-bit (or wider) mantissa of long
    double holds pos * freq to 2^-64 of itself: 2^-33 radians at 2^31."""
    angle = np.asarray(pos)[..., None].astype(np.longdouble) * np.asarray(freqs).astype(np.longdouble)
    return (amplitude * np.cos(angle)).astype(np.float64), (amplitude * np.sin(angle)).astype(np.float64)


def turn(x, pos, freqs, offset=0, interleaved=False, amplitude=1.0, inverse=False):
    """(y, sum of the magnitudes of y's terms) for x fp64 [..., h, d], pos [...]."""
    rot = 2 * len(freqs)
    c, s = factors(pos, freqs, amplitude)
    c, s = c[..., None, :], (-s if inverse else s)[..., None, :]
    one = slice(offset, offset + rot, 2) if interleaved else slice(offset, offset + rot // 2)
    two = slice(offset + 1, offset + rot, 2) if interleaved else slice(offset + rot // 2, offset + rot)
    y, mag = x.copy(), np.abs(x)
    x1, x2 = x[..., one], x[..., two]
    with np.errstate(invalid="ignore"):
        y[..., one], y[..., two] = x1 * c - x2 * s, x2 * c + x1 * s
        mag[..., one] = mag[..., two] = amplitude * (np.abs(x1) + np.abs(x2))
    return y, mag
