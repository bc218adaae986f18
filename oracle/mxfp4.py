"""MXFP4 rows (the OCP microscaling format with e2m1 elements): quantiser, values and product.

A block is 32 columns with one scale byte (a power of two, biased by 127; 255 is NaN) and 4-bit
codes.  The quantiser works on whole numbers: a code is found by comparing |x| / 2^e, exact in
fp64, with the halfway points between the eight magnitudes.
"""

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
HALFWAY = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2


def blocks(k):
    return -(-k // BLOCK)


def encode(a):
    """Codes 0..15 of fp64 values already divided by their scale: nearest, halfway to the even code."""
    m = np.abs(a)
    code = np.zeros(a.shape, np.uint8)
    for i, h in enumerate(HALFWAY):
        code += (m > h) | ((m == h) & (i % 2 == 1))
    return code | (np.signbit(a).astype(np.uint8) << 3)


def scale_byte(amax):
    """e + 127 for the largest magnitude of a block; 255 where it is not finite."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(np.where(np.isfinite(amax) & (amax > 0), amax, 2.0 ** -200))
    s = np.clip(e.astype(np.int64) - 1 - 2 + 127, 0, 254)
    return np.where(np.isfinite(amax), s, 255).astype(np.uint8)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(q):
    return np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def quant(x):
    """(codes uint8 [M, 16 KM], scales uint8 [M, KM]) of real rows [M, K]."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    kb = blocks(K)
    b = np.zeros((M, kb * BLOCK))
    b[:, :K] = x
    b = b.reshape(M, kb, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    s = np.where(bad, 255, scale_byte(np.abs(np.where(np.isfinite(b), b, 0)).max(axis=2, initial=0.0))).astype(np.uint8)
    unit = np.ldexp(1.0, s.astype(np.int64) - 127)[:, :, None]
    with np.errstate(invalid="ignore"):
        codes = encode(np.where(bad[:, :, None], 0.0, b) / unit)
    return pack(codes.reshape(M, kb * BLOCK)), s


def values(q, s, K=None):
    """fp64 values [..., K] of codes and scales."""
    c = unpack(np.asarray(q))
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.asarray(s)
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    v = v * np.repeat(scale, BLOCK, axis=-1)
    return v if K is None else v[..., :K]


def gemm(a, a_s, b, b_s):
    """(product in fp64, bound on an fp32 sum's error): every addition of a sum of K terms errs by at
    most 2^-23 of the sum of the magnitudes (a rounding or a truncation)."""
    A, B = values(a, a_s), values(b, b_s)
    return A @ B.T, A.shape[1] * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T)
