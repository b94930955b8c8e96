"""MXFP4 (microscaled 4-bit floating point) in 64 bits: quantising, reading back and the
products, from the definitions of the OCP Microscaling Formats (MX) Specification v1.0.
numpy only; nothing here is shared with the kernels.

An operand of `rows` rows of K values is (codes, scales): codes (rows, 16 * blocks) bytes,
two e2m1 codes per byte with the even k in the low nibble, blocks = ceil(K / 32); scales
(blocks, rows) bytes, 2^(byte - 127), 255 = NaN.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks_of(K: int) -> int:
    return -(-K // BLOCK)


def nearest_code(a):
    """Code of the e2m1 value nearest to each magnitude a >= 0; of two as near, the even code;
    above 6, 6."""
    a = np.minimum(np.asarray(a, np.float64), 6.0)
    hi = np.searchsorted(E2M1, a)                 # E2M1[hi - 1] < a <= E2M1[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = E2M1[hi] - a, a - E2M1[lo]
    even = np.where(hi % 2 == 0, hi, lo)
    return np.where(up < down, hi, np.where(down < up, lo, even)).astype(np.uint8)


def quantize(x, rule: str = "floor"):
    """(codes, scales) of x (rows, K) along K."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    nb = blocks_of(K)
    v = np.zeros((rows, nb * BLOCK))
    v[:, :K] = x
    v = v.reshape(rows, nb, BLOCK)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    a = np.abs(v).max(axis=2) if nb else np.zeros((rows, 0))
    mant, ex = np.frexp(a)                        # a = mant * 2^ex, mant in [0.5, 1)
    e = ex - 1 - 2
    if rule == "fit":
        e = e + (a > np.ldexp(6.0, e))
    e = np.maximum(np.where(a == 0, -127, e), -127)
    scaled = np.ldexp(v, -e[:, :, None])
    code = nearest_code(np.abs(scaled)) | (np.signbit(v).astype(np.uint8) << 3)
    code = np.where(bad[:, :, None], np.uint8(0), code).reshape(rows, nb * BLOCK)
    scales = np.where(bad, 255, e + 127).astype(np.uint8).T
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), np.ascontiguousarray(scales)


def values(codes, scales, K: int):
    """float64 values (rows, K) of an operand."""
    codes, scales = np.asarray(codes, np.uint8), np.asarray(scales, np.uint8)
    rows = codes.shape[0]
    nib = np.stack([codes & 15, codes >> 4], axis=2).reshape(rows, -1)[:, :K]
    mag = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    byte = scales[:, :rows].T.astype(int)
    f = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return mag * np.repeat(f, BLOCK, axis=1)[:, :K]


def product(a, b):
    """(exact product in 64 bits, sum of magnitudes) of values a (M, K) and b (N, K).  NaN
    wherever a factor of the sum is NaN, whatever the other factor."""
    nan = np.isnan(a).any(axis=1)[:, None] | np.isnan(b).any(axis=1)[None, :]
    a, b = np.nan_to_num(a, nan=0.0, posinf=np.inf, neginf=-np.inf), np.nan_to_num(b, nan=0.0, posinf=np.inf, neginf=-np.inf)
    return np.where(nan, np.nan, a @ b.T), np.abs(a) @ np.abs(b).T
