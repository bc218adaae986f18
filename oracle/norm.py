"""RMS norms around a residual connection in fp64, with bounds on an fp32 evaluation.

``u`` is half a step of fp32 (2^-24).  A row's sum of squares is added up in fewer than 86 steps one
after the other (8 columns, a wave, the waves' sums), each squared term rounded once: 90 u at most;
its root halves that; the division by D, the addition of eps, the root and the reciprocal add
4 u: 1 / rms errs by at most 50 u, relative.
"""

import numpy as np

from . import formats as F

U = 2.0 ** -24
RMS = 50 * U


def inverse_rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def forward(x, w, residual=None, post_w=None, gate=None, scale=1.0, eps=1e-6):
    """(h, bound on h, y, bound on y), fp64, before any rounding to bf16; inputs are exact values."""
    t = np.asarray(x, np.float64)
    dt = np.zeros_like(t)
    if post_w is not None:
        t = t * inverse_rms(t, eps) * post_w
        dt = np.abs(t) * (RMS + 2 * U)
    h, dh = t, dt
    if residual is not None:
        g = 1.0 if gate is None else gate
        h = residual + float(np.float32(scale)) * g * t
        part = np.abs(float(np.float32(scale)) * g * t)
        dh = np.abs(scale * g) * dt + part * U + np.abs(h) * U
        dh = dh * (1 + 2.0 ** -10)
    r = inverse_rms(h, eps)
    y = h * r * w
    norm = np.sqrt((h * h).sum(axis=1, keepdims=True))
    off = np.sqrt((dh * dh).sum(axis=1, keepdims=True)) / np.where(norm > 0, norm, 1.0)
    dy = np.abs(r * w) * dh + np.abs(y) * (RMS + 2 * U + 1.01 * off)
    return h, dh, y, dy * (1 + 2.0 ** -10)


def e4m3_codes(h, w, block=128):
    """e4m3 codes of y = h / rms(h) * w under its blocks' scales max |y| / 448, exactly: 1 / rms cancels, and |y| over
    its scale is compared with the halfway point m of two codes as 448 |h w| with m max |h w|.  For h and w of at most 8
    significant bits (m has 5) all of these are exact in fp64.  A halfway case takes the even code."""
    hw = np.asarray(h, np.float64) * w
    T, D = hw.shape
    nb = -(-D // block)
    a = np.abs(np.pad(hw, ((0, 0), (0, nb * block - D)))).reshape(T, nb, block)
    top = a.max(axis=2, keepdims=True)
    v = F.e4m3_decode(np.arange(127, dtype=np.uint8))
    code = np.zeros(a.shape, np.uint8)
    for i, m in enumerate((v[1:] + v[:-1]) / 2):
        code += (448 * a > m * top) | ((448 * a == m * top) & (i % 2 == 1))
    code = code.reshape(T, nb * block)[:, :D]
    return code | (np.signbit(hw).astype(np.uint8) << 7)


def halfway_rows(T, D, g):
    """(x, w) of at most 5 significant bits, many of whose codes are halfway cases: whole numbers, every second block
    with a largest product of 2 * 448, some values so small that their codes are subnormal."""
    x = g.integers(1, 29, (T, D)).astype(np.float32) * g.choice(np.array([-1, 1], np.float32), (T, D))
    x[g.random((T, D)) < 0.2] *= 2.0 ** -9
    w = g.integers(1, 33, D).astype(np.float32)
    x[:, ::256], w[::256] = 28, 32
    return x, w
