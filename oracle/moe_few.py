"""The routed-expert layer for a few tokens, in fp64, with an error bound.

Activations are not quantised; weights are the stored values times their
scales.  ``layer`` returns the result and, element by element, how far a
computation that sums in fp32, carries h with 16 significant bits and rounds
once to bf16 may be from it:

* each product of n terms: 2^-16 of the sum of the terms' magnitudes (fp32
  summation of up to a few thousand terms stays well below; the matrix
  instruction may align the terms of one step to their largest before adding);
* the gate: SiLU' <= 1.1, the hardware exponential and reciprocal and the split
  of h into two bf16 values: 2^-16 of |h|;
* the final rounding: half a bf16 unit, at most 2^-8 |out| with the terms above.
"""

import numpy as np

from .formats import bf16_to_f32
from .gemm import dequant_weight

EPS = 2.0 ** -16


def weight_f64(q, s):
    """[n, k] values: int8 with row scales, or e4m3 bytes with 128x128 block scales."""
    if q.dtype == np.int8:
        return q.astype(np.float64) * s.astype(np.float64)[:, None]
    return dequant_weight(q, s)


def layer(x_bits, w13, s13, w2, s2, indices, weight_bits):
    """(out fp64 [T, D], bound fp64 [T, D])."""
    x = bf16_to_f32(x_bits).astype(np.float64)
    wt = bf16_to_f32(weight_bits).astype(np.float64)
    E, F = w13.shape[0], w13.shape[1] // 2
    out, err = np.zeros_like(x), np.zeros_like(x)
    for e in range(E):
        t, j = np.nonzero(np.asarray(indices) == e)
        if t.size == 0:
            continue
        A, B = weight_f64(w13[e], s13[e]), weight_f64(w2[e], s2[e])
        gu, mag = x[t] @ A.T, np.abs(x[t]) @ np.abs(A).T
        g, u, dg, du = gu[:, :F], gu[:, F:], EPS * mag[:, :F], EPS * mag[:, F:]
        with np.errstate(over="ignore"):
            silu = g / (1.0 + np.exp(-g))
        h = silu * u
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + EPS * np.abs(h)
        w = wt[t, j][:, None]
        np.add.at(out, t, w * (h @ B.T))
        np.add.at(err, t, np.abs(w) * ((dh + EPS * np.abs(h)) @ np.abs(B).T))
    return out, err + 2.0 ** -8 * (np.abs(out) + err) + 1e-38
