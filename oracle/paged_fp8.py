"""Plain forms of a cache in 8 bits: e4m3 codes in pages and one power of two
for every 16 slots and head.  NumPy, one block at a time; nothing here is shared
with the CUDA side."""
import numpy as np

from oracle import fp8
from oracle import paged_fp64 as P

BLOCK, LOW, HIGH, BIAS = 16, -100, 119, 127


def _value(code):
    s, e, m = code >> 7, code >> 3 & 15, code & 7
    if e == 15 and m == 7:
        return np.nan
    x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -x if s else x


VALUES = np.array([_value(c) for c in range(256)])


def encode(x):
    """Codes of float64 values: nearest, ties to even, at most 448; what is not finite is NaN."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    # e4m3_round ends in float32, which holds every e4m3 value
    return np.where(fine, fp8.e4m3_bits(fp8.e4m3_round(np.where(fine, x, 0))), np.uint8(0x7f)).astype(np.uint8)


def values(codes, scales):
    """What a pool [pages, page, H, d] of codes stands for."""
    s = np.ldexp(1.0, np.minimum(scales, HIGH + BIAS).astype(int) - BIAS)
    return VALUES[codes] * np.repeat(s, BLOCK, axis=1)[..., None]


def exponent(top):
    """The least e with top <= 448 2^e, within [LOW, HIGH]."""
    e = LOW
    while e < HIGH and top > np.ldexp(448.0, e):
        e += 1
    return e


def append(codes, scales, rows, table, lens, cu, page):
    """(codes, scales) with the new tokens' rows [T, H, d] in place."""
    H, d = codes.shape[2:]
    c, s = codes.copy().reshape(-1, H, d), scales.copy().reshape(-1, H)
    for b, L in enumerate(lens):
        n = int(cu[b + 1] - cu[b])
        at = P.slots(table[b], L, page)
        for first in range((L - n) // BLOCK * BLOCK, L, BLOCK) if n else ():
            lo, hi = max(first, L - n), min(first + BLOCK, L)
            blk = at[first] // BLOCK
            for h in range(H):
                x = rows[cu[b] + lo - (L - n):cu[b] + hi - (L - n), h].astype(np.float64)
                a = np.abs(x[np.isfinite(x)])
                e = exponent(a.max() if a.size else 0.0)
                if lo > first:
                    was = min(int(s[blk, h]) - BIAS, HIGH)
                    e = max(e, was)
                    if e > was:
                        old = VALUES[c[at[first:lo], h]]
                        c[at[first:lo], h] = np.where(np.isnan(old), c[at[first:lo], h], encode(np.ldexp(old, was - e)))
                c[at[lo:hi], h] = encode(np.ldexp(x, -e))
                s[blk, h] = e + BIAS
    return c.reshape(codes.shape), s.reshape(scales.shape)
