"""The 8-bit K/V cache's format, from its definition, in float64 NumPy.

A row is d e4m3 codes and one exponent byte E; its values are code * s with s
the fp32 number whose exponent field is E and whose mantissa is 0.  Quantising
takes the smallest power of two s = 2^(E-127), 1 <= E <= 254, with |x| <= 448 s
for the row's finite values, and the e4m3 number nearest to x / s (of two
equally near, the one whose last mantissa bit is 0)."""
from __future__ import annotations

import numpy as np


def e4m3_table():
    """The 256 codes' values: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    no infinities; exponent and mantissa all ones is NaN."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** -9
        else:
            out[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


TABLE = e4m3_table()


def scale_of(exps):
    e = np.asarray(exps).astype(np.int64)
    return np.where(e == 0, 0.0, np.where(e == 255, np.inf, np.exp2(e - 127.0)))


def quantise(x):
    """(codes uint8, exponents uint8) of rows x[..., d]."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    top = np.where(np.isfinite(a), a, 0.0).max(axis=-1)
    exps = np.ones(top.shape, np.int64)
    for p in range(-126, 127):            # the smallest s is the first that is large enough
        exps += top > 448.0 * 2.0 ** p
    with np.errstate(invalid="ignore"):
        y = x * np.exp2(127.0 - exps)[..., None]
    mags = TABLE[:127]                    # 0 .. 448, ascending with the code
    ay = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(mags, ay), 1, 126)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        up, down = mags[hi] - ay, ay - mags[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(y), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8), exps.astype(np.uint8)


def values(codes, exps):
    """float64 rows of codes [b, m, g, d] and exponents [b, g, m]."""
    with np.errstate(invalid="ignore"):
        return TABLE[codes] * np.moveaxis(scale_of(exps), 1, 2)[..., None]
