"""8-bit codes with a scale a group, and their product (oracle side).

The codes are formed in binary64, which decides every one of them rightly:
|x| and the scale are binary32 numbers, so |x|/s + r16/65536 is either an
integer exactly (and then both the quotient and the sum are exact in
binary64) or at least 2**-41 away from one, and the two roundings cost less
than 2**-45. ``codes_scalar`` does the same in rational arithmetic.

Test infrastructure only (see the package header).
"""

import math
from fractions import Fraction

import numpy as np

from .stream import random16

TINY = np.float32(2.0 ** -126)


def scale_of(amax):
    """f32(amax / 127) of a binary32 amax, 0 below 2**-126 and NaN when amax
    is not finite. (The binary64 quotient of a 24-bit number by 127 is never
    within its own rounding error of a binary32 tie.)"""
    amax = np.asarray(amax, dtype=np.float32)
    with np.errstate(invalid="ignore"):
        s = (amax.astype(np.float64) / 127.0).astype(np.float32)
    s = np.where(s < TINY, np.float32(0), s)
    return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def quantize(x, transpose=False, rounding="rn", seed=0, step=0, base_index=0):
    """(codes int8, scales f32) of a matrix of binary32 values; transposed
    codes for transpose=True."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    share = None
    if rounding == "sr":
        pos = (np.uint64(int(base_index) & 0xFFFFFFFFFFFFFFFF)
               + np.arange(rows * cols, dtype=np.uint64)).reshape(rows, cols)
        share = random16(pos, seed, step).astype(np.float64) / 65536.0
    if transpose:
        x = x.T
        share = None if share is None else share.T
    if x.shape[1] == 0:
        return np.zeros(x.shape, np.int8), np.zeros(x.shape[0], np.float32)
    with np.errstate(invalid="ignore"):
        amax = np.max(np.where(np.isnan(x), np.float32(np.inf), np.abs(x)), axis=1)
    s = scale_of(amax)
    live = s > 0
    div = np.where(live, s, np.float32(1)).astype(np.float64)[:, None]
    t = np.where(live[:, None], np.abs(np.where(np.isfinite(x), x, 0)).astype(np.float64) / div, 0.0)
    q = np.rint(t) if share is None else np.floor(t + share)
    q = np.where(live[:, None], np.minimum(q, 127.0), 0.0)
    return (np.sign(np.where(np.isfinite(x), x, 0)) * q).astype(np.int8), s


def code_scalar(x, s, r16=None):
    """One code in rational arithmetic (x finite, s > 0; r16 None: nearest, even)."""
    t = abs(Fraction(float(x))) / Fraction(float(s))
    q = round(t) if r16 is None else math.floor(t + Fraction(int(r16), 65536))
    q = min(q, 127)
    return -q if x < 0 else q


def gemm_f32(a, b, scale_a, scale_b):
    """(f32(sum a b) * sa) * sb in binary32; the sums exact."""
    # (binary64 holds every partial sum of int8 products exactly)
    acc = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T
    with np.errstate(over="ignore", invalid="ignore"):
        v = acc.astype(np.float32) * np.asarray(scale_a, np.float32)[:, None]
        return v * np.asarray(scale_b, np.float32)[None, :]
