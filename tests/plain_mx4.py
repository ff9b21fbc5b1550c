"""Plain microscaled 4-bit rows on numpy arrays in binary64 (test helper),
written from the formulas in include/qk.h."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest(u):
    """Codes 0 .. 7 of magnitudes u in units of their scale: the nearest level,
    ties to the even code, at most 6."""
    hi = np.minimum(np.searchsorted(LEVELS, u), 7)
    lo = np.maximum(hi - 1, 0)
    down, up = u - LEVELS[lo], LEVELS[hi] - u
    lower = (down < up) | ((down == up) & (lo % 2 == 0))
    return np.where(lower, lo, hi).astype(np.uint8)


def quantise(x):
    """(code per value, scale byte per block) of rows of values."""
    x = np.asarray(x, np.float64)
    v = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[..., None], 0.0, v)
    top = np.abs(v).max(2, initial=0.0)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    code = nearest(np.abs(v) * 2.0 ** -e[..., None].astype(np.float64)) | (np.signbit(v).astype(np.uint8) << 3)
    return code.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(q):
    return np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)


def values(q, scale):
    """What packed codes and scale bytes stand for, binary64."""
    code = unpack(q)
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = 2.0 ** (scale.astype(np.float64) - 127)
    s[scale == 255] = np.nan
    return v * np.repeat(s, 32, 1)
