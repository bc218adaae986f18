"""int8 rows with one scale each: quantiser, product, and the gated form.

``row_quant`` follows the definition's fp32 steps one by one (NumPy's float32
operations are correctly rounded), so codes and scales can be compared bit
for bit; ``gemm`` sums in 64-bit integers and applies the definition's two
fp32 multiplications and the rounding to bf16.
"""

import numpy as np

from .formats import bf16_to_f32, f32_to_bf16

AMAX_FLOOR = np.float32(2.0 ** -100)


def row_quant(x):
    """(codes int8 [M, K], scales fp32 [M]) of fp32 rows (bf16 rows are exact in fp32)."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=1, initial=0.0).astype(np.float32)
    amax = np.maximum(amax, AMAX_FLOOR)
    inv = np.float32(127) / amax
    return np.rint(x * inv[:, None]).astype(np.int8), amax / np.float32(127)


def silu_mul(g_bits, u_bits):
    """SiLU(g) * u in fp64 of bf16 bit patterns."""
    g = bf16_to_f32(g_bits).astype(np.float64)
    u = bf16_to_f32(u_bits).astype(np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def gemm(a, a_s, b, b_s):
    """bf16 bits [M, N]; the integer sum is exact (float64 matmul of whole numbers below 2^53)."""
    acc = a.astype(np.float64) @ b.astype(np.float64).T
    scale = np.asarray(a_s, np.float32)[:, None] * np.asarray(b_s, np.float32)[None, :]
    return f32_to_bf16(acc.astype(np.float32) * scale)


def linear(x_bits, b, b_s):
    a, a_s = row_quant(bf16_to_f32(x_bits))
    return gemm(a, a_s, b, b_s)
