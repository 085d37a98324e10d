"""AdamW with fp32 or 8-bit moments, restated plainly in fp64.

8-bit moments: blocks of 128 elements share E = 127 + floor(log2(max)) in [16, 254]; a code's
value is c u below 8 and (8 + c % 8) 2^(c // 8 - 1) u from there on, u = 2^(E - 127 - 17) for the
signed first moment (bit 7 the sign) and 2^(E - 127 - 33) for the second.
"""

import math

import numpy as np

from . import philox

BLOCK = 128
PURPOSE_STATE = 4


def _unit(E, signed):
    return 2.0 ** (np.asarray(E, dtype=np.float64) - (144 if signed else 160))


def _blocks(a):
    a = np.asarray(a, dtype=np.float64)
    pad = -len(a) % BLOCK
    return np.concatenate([a, np.zeros(pad)]).reshape(-1, BLOCK)


def magnitudes(signed):
    """Values of all magnitude codes in units of u."""
    c = np.arange(128 if signed else 256)
    return np.where(c < 8, c, (8 + c % 8) * 2.0 ** (np.maximum(c // 8, 1) - 1))


def decode(codes, E, signed):
    n = len(codes)
    c = np.asarray(codes, dtype=np.int64)
    mag = magnitudes(signed)[c & 127 if signed else c]
    if signed:
        mag = np.where(c > 127, -mag, mag)
    return mag * np.repeat(_unit(E, signed), BLOCK)[:n]


def encode(x, signed, field=None):
    """(codes, E) of the fp64 values x; field: 16 random bits an element, or None for nearest."""
    n = len(x)
    b = _blocks(x)
    bad = ~np.isfinite(b)
    mag = np.where(bad, 0.0, np.abs(b))
    top = mag.max(axis=1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1, -111)
    E = np.clip(e, -111, 127) + 127
    t = mag / _unit(E, signed)[:, None]
    octave = np.maximum(np.frexp(t)[1] - 4, 0)          # t < 16: the lowest two octaves, step 1
    octave = np.where(t > 0, octave, 0)
    s = t / 2.0 ** octave
    if field is None:
        r = np.rint(s)
    else:
        f = np.concatenate([np.asarray(field, dtype=np.float64), np.zeros(-n % BLOCK)]).reshape(-1, BLOCK)
        r = np.floor(s + (f + 0.5) / 65536.0)
    c = np.minimum(r + 8 * octave, 127 if signed else 255).astype(np.int64)
    if signed:
        c = c + 128 * ((b < 0) & (c > 0))
    else:
        c = np.where((mag > 0) & (c == 0), 1, c)
    c = np.where(bad, 0, c)
    return c.reshape(-1)[:n].astype(np.uint8), E.astype(np.uint8)


def words(seed, tensor_id, sub, step, n):
    """The 32-bit word of each element: counter element / 4, word element % 4."""
    return philox.element_words(seed, philox.tag(tensor_id, PURPOSE_STATE, sub), step, n)


def moments(m, v, g, b1, b2):
    """The new moments in fp64, every operation rounded, in the order that the codes are defined by."""
    g = np.asarray(g, dtype=np.float64)
    return b1 * m + (1.0 - b1) * g, b2 * v + (1.0 - b2) * (g * g)


def parameter(p, m, v, t, lr, b1, b2, eps, wd):
    with np.errstate(invalid="ignore", divide="ignore"):
        return np.asarray(p, np.float64) * (1 - lr * wd) - lr / (1 - b1 ** t) * (m / (np.sqrt(v) / math.sqrt(1 - b2 ** t) + eps))
