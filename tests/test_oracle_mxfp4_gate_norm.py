"""CPU pins of the MXFP4, gate and norm oracles against closed forms, brute force and invariants."""

import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import gate as GT
from oracle import mxfp4 as MX
from oracle import norm as NM


def brute_code(v):
    """Nearest of the eight magnitudes by exact distances, halfway to the even code."""
    a = abs(Fraction(float(v)))
    best = min(range(8), key=lambda c: (abs(Fraction(float(MX.MAGNITUDES[c])) - a), c % 2))
    return best | (8 if np.signbit(v) else 0)


def test_codes_against_exact_distances():
    g = np.random.default_rng(0)
    v = np.concatenate([MX.MAGNITUDES, MX.HALFWAY, np.nextafter(MX.HALFWAY, 0), np.nextafter(MX.HALFWAY, 9),
                        [7.0, 7.999, 100.0, 1e-300], g.uniform(0, 8, 500)])
    v = np.concatenate([v, -v])
    assert MX.encode(v).tolist() == [brute_code(x) for x in v]


def test_scale_of_powers_and_neighbours():
    for e in (-149, -126, -125, -124, -20, 0, 1, 100, 127):
        top = np.float32(2.0 ** e) if e >= -149 else 0
        want = max(e - 2, -127) + 127
        assert MX.scale_byte(top) == want
        assert MX.scale_byte(np.nextafter(top, np.float32(np.inf))) == want
    assert MX.scale_byte(0.0) == 0 and MX.scale_byte(np.inf) == 255 and MX.scale_byte(np.nan) == 255


@pytest.mark.parametrize("K", [1, 31, 32, 33, 96, 100])
def test_round_trip(K):
    """Values that the format holds come back; others are within half a step of a block's scale."""
    g = np.random.default_rng(K)
    x = g.standard_normal((7, K)) * np.exp2(g.integers(-40, 40, (7, 1)))
    q, s = MX.quant(x)
    assert q.shape == (7, 16 * MX.blocks(K)) and s.shape == (7, MX.blocks(K))
    v = MX.values(q, s, K)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), MX.BLOCK, axis=1)[:, :K]
    assert np.all(np.abs(v - x) <= np.where(np.abs(x) < 6 * unit, 1.0, 2.0) * unit)
    q2, s2 = MX.quant(v)
    assert np.array_equal(MX.values(q2, s2, K), v)
    assert not MX.unpack(q)[:, K:].any()


def test_bad_blocks():
    x = np.ones((3, 64))
    x[0, 5], x[1, 40], x[2, 63] = np.nan, np.inf, -np.inf
    _, s = MX.quant(x)
    assert s.tolist() == [[255, 125], [125, 255], [125, 255]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gate_against_enumeration(score):
    """The chosen set is the best of all sets, in order, for small cases with ties and missing experts."""
    g = np.random.default_rng(1)
    for trial in range(40):
        E, k = 6, 3
        x = g.integers(-2, 3, (1, E)).astype(np.float32)
        x[0, g.integers(0, E)] = -np.inf
        idx, w = GT.gate(x, k, score=score, scale=2.0)
        sc = GT.scores(x, score)[0]
        can = [e for e in range(E) if x[0, e] != -np.inf]
        best = max(itertools.permutations(can, k), key=lambda p: ([sc[e] for e in p], [-e for e in p]))
        assert idx[0].tolist() == list(best)
        assert abs(w.sum() - 2.0) < 1e-12


def test_gate_scores_against_torch():
    x = torch.linspace(-30, 30, 301, dtype=torch.float64)[None]
    assert np.array_equal(GT.scores(x.numpy(), "sigmoid"), torch.sigmoid(x).float().numpy())
    np.testing.assert_allclose(GT.scores(x.numpy(), "softmax"), torch.softmax(x, 1).float().numpy(), rtol=2 ** -23)


def test_gate_groups():
    x = np.array([[3.0, 0.0, 2.0, 2.0, 2.5, -np.inf]], np.float32)   # groups of 2
    assert GT.gate(x, 2, groups=3, top_groups=1)[0].tolist() == [[0, 1]]
    b = np.zeros(6, np.float32)                                      # with a bias the two best count
    assert GT.gate(x, 2, bias=b, groups=3, top_groups=1)[0].tolist() == [[2, 3]]
    x[0, 0] = -np.inf
    assert GT.gate(x, 4, groups=3, top_groups=2)[0].tolist() == [[4, 2, 3, -1]]
    assert GT.gate(np.full((1, 6), -np.inf, np.float32), 2)[0].tolist() == [[-1, -1]]


def test_norm_invariants():
    g = np.random.default_rng(2)
    x, w = g.standard_normal((5, 33)), g.standard_normal(33)
    h, dh, y, dy = NM.forward(x, np.ones(33), eps=0.0)
    assert np.array_equal(h, x) and not dh.any()
    np.testing.assert_allclose((y * y).mean(axis=1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(NM.forward(3.5 * x, w, eps=0.0)[2], NM.forward(x, w, eps=0.0)[2], rtol=1e-12)
    r, gate = g.standard_normal((5, 33)), g.standard_normal((5, 33))
    h2 = NM.forward(x, w, residual=r, post_w=w, gate=gate, scale=0.5, eps=0.0)[0]
    np.testing.assert_allclose(h2, r + 0.5 * gate * (x / np.sqrt((x * x).mean(1, keepdims=True)) * w), rtol=1e-12)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (33,), torch.from_numpy(w), 1e-6).numpy()
    np.testing.assert_allclose(NM.forward(x, w)[2], ref, rtol=1e-12)


def test_norm_codes_against_fractions():
    """Codes of the exact quotient, and that a 32-bit evaluation gives others on the same rows: what a kernel is
    compared with on them tells the two apart."""
    x, w = NM.halfway_rows(3, 300, np.random.default_rng(3))
    codes = NM.e4m3_codes(x, w)
    values = [Fraction(float(v)) for v in F.e4m3_decode(np.arange(127, dtype=np.uint8))]
    ties = 0
    for t in range(3):
        for b in range(0, 300, 128):
            hw = [Fraction(float(x[t, k])) * Fraction(float(w[k])) for k in range(b, min(300, b + 128))]
            top = max(abs(v) for v in hw)
            for k, v in enumerate(hw):
                q = 448 * abs(v) / top
                best = min(range(127), key=lambda c: (abs(values[c] - q), c % 2))
                assert codes[t, b + k] == best | (128 if v < 0 else 0)
                near = sorted(abs(c - q) for c in values)
                ties += near[0] == near[1]
    assert ties > 45                    # one in twenty
    x, w = NM.halfway_rows(64, 1024, np.random.default_rng(4))
    y = x * np.float32(NM.inverse_rms(x.astype(np.float64), 1e-6)).astype(np.float32) * w
    b = y.reshape(64, 8, 128)
    s = np.abs(b).max(axis=2, keepdims=True) / np.float32(448)
    off = F.e4m3_encode((b / s).reshape(64, 1024)) != NM.e4m3_codes(x, w)
    assert off.sum() > 100
