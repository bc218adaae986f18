"""GPU checks of the choice of experts: indices exactly, weights within their roundings.

A weight is a score over a sum of at most 16 scores times the scale, each step one fp32 rounding
(at most 18 of 2^-24), rounded once more to bf16 (2^-8).  Below 2^-126 bf16's values are 2^-133
apart, so that rounding is off by up to 2^-134 there however small the value; the fp32 steps,
2^-149 apart there, by at most 3 half steps.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as ds
from block_scaled_fp8_act_amd import inputs as I
from oracle import gate as GT

from gpu_helpers import bf16_to_f64, host_bits16

pytestmark = pytest.mark.gpu

CID = 130


def check(x, k, bias=None, dtype=torch.float32, **kw):
    xt = torch.from_numpy(x).to(dtype)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, w = ds.moe_gate(xt.cuda(), k, bias=b, **kw)
    ri, rw = GT.gate(xt.float().numpy(), k, bias=bias, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    got = bf16_to_f64(host_bits16(w))
    assert np.all(np.abs(got - rw) <= np.abs(rw) * (2.0 ** -8 + 20 * 2.0 ** -24) + 2.0 ** -134 + 2.0 ** -148)
    return idx, w


CASES = [(1, 8, 2, 1, 1), (5, 60, 4, 1, 1), (33, 64, 6, 8, 3), (17, 65, 8, 5, 2), (40, 128, 16, 4, 4), (9, 200, 3, 10, 1),
         (64, 256, 8, 8, 4), (3, 257, 1, 1, 1), (12, 384, 8, 64, 9), (7, 512, 10, 2, 1), (6, 1000, 16, 40, 7),
         (4, 1024, 8, 16, 4), (3, 1500, 5, 50, 50), (2, 4096, 16, 64, 3), (4, 7, 7, 1, 1), (300, 16, 1, 16, 2), (1, 1, 1, 1, 1)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top", CASES)
def test_choice(T, E, k, groups, top, bias, score):
    g = I.rng(CID, T * E + groups)
    x = (1.5 * g.standard_normal((T, E)) + 0.5 * g.standard_normal(E)).astype(np.float32)
    b = (0.1 * g.standard_normal(E)).astype(np.float32) if bias else None
    check(x, k, b, score=score, groups=groups, top_groups=top, scale=2.5)
    check(x, k, b, dtype=torch.bfloat16, score=score, groups=groups, top_groups=top, renormalize=False, scale=1.0)


# groups that begin inside a lane's experts: larger than a lane holds, and smaller, for a wave and a quarter
# of one per token and every number of experts a lane takes
UNEVEN = [(300, 250, 6, 5, 2), (9000, 250, 6, 5, 2), (40, 130, 4, 13, 3), (8200, 60, 4, 20, 5), (8200, 126, 5, 7, 2),
          (8195, 90, 3, 30, 9), (70, 500, 8, 20, 7), (30, 420, 8, 60, 11), (50, 1000, 8, 40, 7), (20, 3900, 8, 60, 5),
          (12, 2016, 16, 63, 6), (9, 4090, 8, 5, 3)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top", UNEVEN)
def test_groups_that_begin_inside_a_lane(T, E, k, groups, top, bias, score):
    test_choice(T, E, k, groups, top, bias, score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", [(6, 1), (64, 8), (130, 13), (256, 4)])
def test_ties_and_saturation(E, groups, score):
    """Few distinct logits, some so large that their fp32 scores are equal: the lowest index first."""
    g = I.rng(CID, E)
    x = g.choice(np.array([-60.0, -1.0, 0.0, -0.0, 0.5, 17.5, 40.0, 90.0], np.float32), (50, E))
    check(x, min(5, E), score=score, groups=groups, top_groups=max(1, groups // 2))
    b = g.choice(np.array([-0.5, 0.0, 0.25, 1e-9], np.float32), E)
    check(x, min(5, E), b, score=score, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_missing_experts(bias, score):
    """Logits and biases of -inf, the type's lowest value, tokens with fewer than k experts and with none."""
    g = I.rng(CID, 7)
    T, E = 40, 24
    x = g.standard_normal((T, E)).astype(np.float32)
    x[g.random((T, E)) < 0.5] = -np.inf
    x[3], x[11, 1:] = -np.inf, -np.inf
    x[5] = np.finfo(np.float32).min
    x[6, ::2] = np.finfo(np.float32).min
    b = None
    if bias:
        b = (0.1 * g.standard_normal(E)).astype(np.float32)
        b[4] = -np.inf
        b[9] = np.finfo(np.float32).min
        b[10] = np.finfo(np.float32).max
    for groups, top in ((1, 1), (6, 2), (24, 7), (2, 1)):
        idx, w = check(x, 6, b, score=score, groups=groups, top_groups=top)
        assert (idx[3] == -1).all() and not w[3].any()
        # the routed-expert layer takes such slots as no expert
        off, _, rows = ds.moe_route(idx, E)
        assert torch.equal(rows < 0, idx < 0) and int(off[-1]) == int((idx >= 0).sum())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups,top", [(40, 24, 6, 4), (40, 250, 5, 3), (8200, 60, 4, 3), (8193, 126, 7, 4), (30, 130, 13, 9)])
def test_groups_masked_by_the_lowest_value(T, E, groups, top, score):
    """Biases of the type's lowest value: a group's two best keys add up to -inf, and the group still comes before
    those whose experts are all missing; tokens without whole groups."""
    g = I.rng(CID, 9)
    size = E // groups
    x = g.standard_normal((T, E)).astype(np.float32)
    b = (0.1 * g.standard_normal(E)).astype(np.float32)
    b[(groups - 1) * size:] = np.finfo(np.float32).min
    for t in range(T):
        gone = g.permutation(groups - 1)[:int(g.integers(0, groups))]
        for q in gone:
            x[t, q * size:(q + 1) * size] = -np.inf
    x[1, g.random(E) < 0.7] = -np.inf
    check(x, 4, b, score=score, groups=groups, top_groups=top)


def test_nan_shows_and_stays_in_its_row():
    g = I.rng(CID, 8)
    x = g.standard_normal((9, 40)).astype(np.float32)
    clean = ds.moe_gate(torch.from_numpy(x).cuda(), 4, groups=4, top_groups=2)
    x[2, 17], x[4] = np.nan, np.nan
    x[6, 3] = np.inf
    for score in ("sigmoid", "softmax"):
        idx, w = (v.cpu() for v in ds.moe_gate(torch.from_numpy(x).cuda(), 4, score=score))
        bad = [2, 4] + ([6] if score == "softmax" else [])
        assert torch.isnan(w[bad]).all() and not torch.isnan(w[[r for r in range(9) if r not in bad]]).any()
        assert ((idx >= 0) & (idx < 40)).all() and all(len(set(r.tolist())) == 4 for r in idx)
    idx, w = ds.moe_gate(torch.from_numpy(x).cuda(), 4, groups=4, top_groups=2)
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(idx[keep], clean[0][keep]) and torch.equal(w[keep], clean[1][keep])


# a group's keys in several lanes, in one, and in parts of lanes; a wave and a quarter of one per token
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,groups", [(3, 64, 2), (3, 256, 8), (3, 384, 6), (3, 250, 5), (3, 1000, 40), (3, 2048, 64),
                                        (8195, 256, 8), (8195, 250, 5), (8195, 60, 20), (8195, 96, 2)])
def test_group_of_nan_comes_before_a_masked_one(T, E, groups, bias):
    """Experts whose keys are NaN are available: a group of them is kept before groups whose experts are all missing,
    and after one with a number."""
    size = E // groups
    x = torch.full((T, E), -float("inf"))
    x[0, size:2 * size] = float("nan")                  # the only group with experts
    x[1, -size:] = float("nan")
    x[2, :size] = float("nan")                          # one NaN group, one of numbers
    x[2, size:2 * size] = 0.25
    b = torch.zeros(E, device="cuda") if bias else None
    idx, w = (v.cpu() for v in ds.moe_gate(x.cuda(), 2, bias=b, groups=groups, top_groups=1))
    for row, first in ((0, size), (1, E - size), (2, size)):
        assert idx[row].tolist() == [first, first + 1], row
        assert torch.isnan(w[row]).all()
    assert (idx[3:] == -1).all() and not w[3:].any()
    # a bias of NaN does the same to an expert of every token
    if bias:
        b[size:2 * size] = float("nan")
        x[:] = -float("inf")
        x[:, size:2 * size] = 0.5
        idx, w = (v.cpu() for v in ds.moe_gate(x.cuda(), 2, bias=b, groups=groups, top_groups=1))
        assert (idx == torch.tensor([size, size + 1], dtype=torch.int32)).all() and torch.isnan(w).all()


def test_strides_and_out():
    g = I.rng(CID, 9)
    x = g.standard_normal((13, 100)).astype(np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        big = torch.zeros((13, 120), dtype=dtype, device="cuda")
        big[:, 3:103] = torch.from_numpy(x).to(dtype).cuda()
        idx = torch.full((13, 9), 5, dtype=torch.int32, device="cuda")
        w = torch.full((13, 11), 5.0, dtype=torch.bfloat16, device="cuda")
        ds.moe_gate(big[:, 3:103], 6, out=(idx[:, 2:8], w[:, 1:7]))
        ri, rw = ds.moe_gate(big[:, 3:103].contiguous(), 6)
        assert torch.equal(idx[:, 2:8], ri) and torch.equal(w[:, 1:7], rw)
        assert (idx[:, [0, 1, 8]] == 5).all() and (w[:, [0, 7, 8, 9, 10]] == 5).all()


def test_no_tokens():
    idx, w = ds.moe_gate(torch.empty((0, 8), device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)


def test_graph():
    x = torch.zeros((70, 64), device="cuda")
    out = (torch.empty((70, 6), dtype=torch.int32, device="cuda"), torch.empty((70, 6), dtype=torch.bfloat16, device="cuda"))

    def step():
        ds.moe_gate(x, 6, groups=8, top_groups=4, out=out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(4):
        x.copy_(torch.from_numpy(I.rng(CID, 50 + seed).standard_normal((70, 64)).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out))
        assert np.array_equal(got[0].cpu().numpy(), GT.gate(x.cpu().numpy(), 6, groups=8, top_groups=4)[0])


def test_refusals():
    x = torch.zeros((4, 64), device="cuda")
    for bad in (lambda: ds.moe_gate(x, 0), lambda: ds.moe_gate(x, 17), lambda: ds.moe_gate(x, 65), lambda: ds.moe_gate(x, 2, groups=7),
                lambda: ds.moe_gate(x, 2, groups=8, top_groups=9), lambda: ds.moe_gate(x, 9, groups=8, top_groups=1),
                lambda: ds.moe_gate(x, 2, score="relu"), lambda: ds.moe_gate(x.half(), 2), lambda: ds.moe_gate(x[0], 2),
                lambda: ds.moe_gate(x.cpu(), 2), lambda: ds.moe_gate(x, 2, bias=torch.zeros(63, device="cuda")),
                lambda: ds.moe_gate(x, 2, bias=torch.zeros(64, device="cuda").double()), lambda: ds.moe_gate(x.t(), 2),
                lambda: ds.moe_gate(x, 2, out=(torch.zeros((4, 2), device="cuda"), torch.zeros((4, 2), device="cuda")))):
        with pytest.raises(ds.Dsfp8Error):
            bad()


@pytest.mark.parametrize("k", [-1, 0, 17, 2.0, None, "2"])
def test_refused_numbers_of_experts(k):
    with pytest.raises(ds.Dsfp8Error):
        ds.moe_gate(torch.zeros((4, 64), device="cuda"), k)
    with pytest.raises(ds.Dsfp8Error):
        ds.moe_gate(torch.zeros((4, 64), device="cuda"), k, out=(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), None))
