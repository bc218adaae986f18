"""RMS norms around a residual connection in fp64, with bounds on an fp32 evaluation.

``u`` is half a step of fp32 (2^-24).  A row's sum of squares is added up in fewer than 86 steps one
after the other (8 columns, a wave, the waves' sums), each squared term rounded once: 90 u at most;
its root halves that; the division by D, the addition of eps, the root and the reciprocal add
4 u: 1 / rms errs by at most 50 u, relative.
"""

import numpy as np

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
