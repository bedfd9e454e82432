"""Plain NumPy statement of MXFP4 rows: E2M1 codes (a sign, two exponent bits,
one mantissa bit) and one E8M0 scale byte per 32 columns, as the OCP
Microscaling Formats specification v1.0 describes the format (sections 5.3.3
and 6.3: shared exponent floor(log2 max) less the largest element exponent,
elements rounded to nearest even, saturating).

Values are fp64 arrays of what the device holds; every step is exact there.
"""
import numpy as np

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes uint8 [M, K] in 0 .. 15, scales uint8 [M, K / 32])."""
    M, K = x.shape
    g = x.reshape(M, K // BLOCK, BLOCK)
    mag = np.abs(g)
    bad = ~np.all(np.isfinite(mag), axis=-1)
    top = np.where(bad, 0.0, np.max(np.where(np.isfinite(mag), mag, 0.0), axis=-1))
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)
    s = np.clip(e + 127, 0, 254)
    a = np.where(bad[..., None], 0.0, mag) / np.ldexp(1.0, s - 127)[..., None]
    # the nearest value; the even code where two are as near
    d = np.abs(a[..., None] - VALUES)
    near = d == d.min(axis=-1, keepdims=True)
    first = near.argmax(axis=-1)
    both = near.sum(axis=-1) == 2
    c = np.where(both & (first % 2 == 1), first + 1, first)
    c = np.where(bad[..., None], 0, c + 8 * np.signbit(g))
    return c.reshape(M, K).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def dequantize(codes, scales):
    """The fp64 values."""
    v = np.where(codes >= 8, -1.0, 1.0) * VALUES[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def pack(codes):
    """uint32 words [M, K / 8], code k at bits 4 (k % 8)."""
    M, K = codes.shape
    c = codes.reshape(M, K // 8, 8).astype(np.uint32)
    return np.bitwise_or.reduce(c << (4 * np.arange(8, dtype=np.uint32)), axis=-1)
