"""Pins of the int8 oracle and of the few-token layer's (no GPU)."""

from fractions import Fraction

import numpy as np
import pytest

from block_scaled_fp8_act_amd import inputs as I
from oracle import formats as F
from oracle import int8 as Q8
from oracle import moe as MOE
from oracle import moe_few as MF
from oracle import quant as Q


def test_row_quant_hand_worked():
    # a = 254, 127 / a = 0.5 exactly: halves go to the even integer
    y, s = Q8.row_quant(np.array([[254.0, 1.0, 3.0, 5.0, -1.0, -3.0, 0.0]], np.float32))
    assert y.tolist() == [[127, 0, 2, 2, 0, -2, 0]] and s[0] == np.float32(2.0)
    y, s = Q8.row_quant(np.zeros((2, 5), np.float32))
    assert not y.any() and np.all(s == np.float32(2.0 ** -100) / np.float32(127))
    y, s = Q8.row_quant(np.zeros((3, 0), np.float32))
    assert y.shape == (3, 0) and s.shape == (3,)


def test_row_quant_is_exact_rational_steps():
    g = np.random.default_rng(0)
    x = g.standard_normal((4, 50)).astype(np.float32) * np.float32(3)
    y, s = Q8.row_quant(x)
    for m in range(4):
        a = Fraction(float(np.abs(x[m]).max()))
        inv = np.float32(float(Fraction(127) / a))          # one rounding to double, one to float
        for k in range(50):
            p = np.float32(np.float64(x[m, k]) * np.float64(inv))   # exact in double, rounded once
            assert y[m, k] == int(round(float(p)))
        assert abs(Fraction(float(s[m])) * 127 / a - 1) < Fraction(1, 1 << 23)
    assert np.abs(y).max(axis=1).tolist() == [127] * 4
    assert np.all(np.abs(y * s[:, None].astype(np.float64) - x) <= s[:, None] * 0.5001)


def test_gemm_against_integers():
    g = np.random.default_rng(1)
    a = g.integers(-127, 128, (5, 33), dtype=np.int8)
    b = g.integers(-127, 128, (7, 33), dtype=np.int8)
    one = Q8.gemm(a, np.ones(5, np.float32), b, np.ones(7, np.float32))
    ref = a.astype(np.int64) @ b.astype(np.int64).T
    assert np.array_equal(one, F.f32_to_bf16(ref.astype(np.float32)))
    scaled = Q8.gemm(a, np.full(5, 0.5, np.float32), b, np.full(7, 4.0, np.float32))
    assert np.array_equal(F.bf16_to_f32(scaled), 2 * F.bf16_to_f32(one))
    assert not Q8.gemm(a[:, :0], np.ones(5, np.float32), b[:, :0], np.ones(7, np.float32)).any()


def test_silu_mul_matches_definition():
    g = I.to_bf16_bits(np.array([0.0, 1.0, -1.0, 30.0, -200.0], np.float32))
    u = I.to_bf16_bits(np.full(5, 2.0, np.float32))
    v = Q8.silu_mul(g, u)
    assert v[0] == 0 and abs(v[1] - v[2] - 2.0) < 1e-15 and abs(v[3] - 60) < 1e-9 and abs(v[4]) < 1e-80


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_layer_one_expert_is_the_dense_network(fmt):
    g = np.random.default_rng(2)
    D, Fh = 40, 24
    if fmt == "int8":
        w13, s13 = Q8.row_quant(g.standard_normal((2 * Fh, D)))
        w2, s2 = Q8.row_quant(g.standard_normal((D, Fh)))
    else:
        w13, s13 = Q.weight_quant(g.standard_normal((2 * Fh, D)).astype(np.float32))
        w2, s2 = Q.weight_quant(g.standard_normal((D, Fh)).astype(np.float32))
    x = I.to_bf16_bits(g.standard_normal((3, D)).astype(np.float32))
    one = I.to_bf16_bits(np.array([[1.0, 1.0], [0.5, 0.25], [1.0, 2.0]], np.float32))
    idx = np.array([[0, 7], [0, 0], [-1, 1]], np.int32)      # outside [0, 1): nothing
    out, bound = MF.layer(x, w13[None], s13[None], w2[None], s2[None], idx, one)
    xf = F.bf16_to_f32(x).astype(np.float64)
    A, B = MF.weight_f64(w13, s13), MF.weight_f64(w2, s2)
    gu = xf @ A.T
    y = (gu[:, :Fh] / (1 + np.exp(-gu[:, :Fh])) * gu[:, Fh:]) @ B.T
    assert np.allclose(out, y * np.array([[1.0], [0.75], [0.0]]), rtol=1e-12, atol=0)
    assert np.all(bound > 0) and np.all(out[2] == 0)
    assert np.median(bound[:2] / np.abs(out[:2])) < 0.02


def test_layer_is_near_the_quantised_pipeline():
    """The existing pipeline quantises activations to e4m3; both approximate one layer."""
    g = np.random.default_rng(3)
    T, E, k, D, Fh = 6, 4, 2, 256, 128
    q13 = [Q.weight_quant((0.05 * g.standard_normal((2 * Fh, D))).astype(np.float32)) for _ in range(E)]
    q2 = [Q.weight_quant((0.05 * g.standard_normal((D, Fh))).astype(np.float32)) for _ in range(E)]
    w13, s13 = (np.stack(v) for v in zip(*q13))
    w2, s2 = (np.stack(v) for v in zip(*q2))
    x = I.to_bf16_bits(g.standard_normal((T, D)).astype(np.float32))
    idx, wb = I.zipf_topk(T, E, k, 1.1)
    ref, _ = MF.layer(x, w13, s13, w2, s2, idx, wb)
    got = F.bf16_to_f32(MOE.moe_forward(x, idx, wb, w13, s13, w2, s2)).astype(np.float64)
    assert np.linalg.norm(got - ref) / np.linalg.norm(ref) < 0.08
