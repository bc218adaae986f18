"""The decode example: routed experts and an int8 shared expert together, eager and as a graph.

Tolerances, element by element: the routed sum within the bound of oracle/moe_few.py.  The shared expert's
up-projection is defined bit for bit.  Its hidden values h are within (|g| + 8) 2^-23 of themselves (the hardware
exponential and reciprocal), the row's maximum and with it the scale likewise, so a code differs by one at most, and
only where the quotient lies within 127 (|g| + max |g| + 18) 2^-23 of a half: |dy| <= sum_f (scale) |w2| over those f,
and (max |g| + 9) 2^-23 of sum |h| |w2| for the scale itself.  Then two roundings to bf16 (the two parts) and one of
their sum, 2^-8 of each."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from block_scaled_fp8_act_amd import inputs as I
from oracle import int8 as Q8
from oracle import moe_few as MF
from oracle import quant as Q
from oracle.formats import bf16_to_f32

from gpu_helpers import bf16_to_f64, dev_bf16, host_bits16

pytestmark = pytest.mark.gpu

CID = 95


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_moe_layer.py")
    spec = importlib.util.spec_from_file_location("decode_moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def shared_expert(x, w13, s13, w2, s2):
    """(fp64 result, error bound) of the int8 shared expert."""
    gu = Q8.linear(x, w13, s13)
    Fh = w2.shape[1]
    h = Q8.silu_mul(gu[:, :Fh], gu[:, Fh:])
    q, qs = Q8.row_quant(h.astype(np.float32))
    y = (q.astype(np.float64) * qs[:, None]) @ MF.weight_f64(w2, s2).T
    g = np.abs(bf16_to_f32(gu[:, :Fh])).astype(np.float64)
    top, scale, mag = g.max(axis=1, keepdims=True), qs[:, None].astype(np.float64), np.abs(MF.weight_f64(w2, s2)).T
    quotient = np.abs(h / scale)
    tie = np.abs(quotient - np.floor(quotient) - 0.5) <= 127 * (g + top + 18) * 2.0 ** -23
    return y, (tie * scale) @ mag + (top + 9) * 2.0 ** -23 * (np.abs(q) * scale) @ mag


@pytest.mark.parametrize("T,E,k,D,Fh,fmt", [(1, 6, 2, 640, 256, "e4m3"), (5, 6, 3, 257, 130, "int8"),
                                            (40, 8, 2, 384, 128, "e4m3")])
def test_layer(T, E, k, D, Fh, fmt):
    quant = Q8.row_quant if fmt == "int8" else Q.weight_quant
    std13, std2 = 1.0 / D ** 0.5, 1.0 / Fh ** 0.5
    q13 = [quant(I.weights_f32((2 * Fh, D), CID, 2 * e, std=std13)) for e in range(E)]
    q2 = [quant(I.weights_f32((D, Fh), CID, 2 * e + 1, std=std2)) for e in range(E)]
    routed = tuple(np.stack(v) for v in zip(*q13)) + tuple(np.stack(v) for v in zip(*q2))
    shared = Q8.row_quant(I.weights_f32((2 * Fh, D), CID, 200, std=std13)) + \
        Q8.row_quant(I.weights_f32((D, Fh), CID, 201, std=std2))
    g = I.rng(CID, 300 + T)
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    wb = I.to_bf16_bits(g.uniform(0.05, 1.0, (T, k)).astype(np.float32))
    x = I.activations((T, D), CID, 400 + T)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    layer = example().DecodeMoeLayer(T, tuple(dev(v) for v in routed), tuple(dev(v) for v in shared))
    args = dev_bf16(x), dev(idx), dev_bf16(wb)
    out = layer(*args).clone()
    r, rb = MF.layer(x, *routed, idx, wb)
    s, sb = shared_expert(x, *shared)
    bound = rb + sb + 2.0 ** -8 * (np.abs(s) + sb + np.abs(r + s) + rb + sb)
    err = np.abs(bf16_to_f64(host_bits16(out)) - (r + s))
    assert np.all(err <= bound), f"{float((err / bound).max()):.3f} of the bound"

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(*args)
    for _ in range(4):
        layer.out.fill_(float("nan"))
        layer.gate_up.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(layer.out, out)
        assert torch.equal(layer(*args), out)


@pytest.mark.parametrize("T,topk", [(1, None), (24, None), (40, 2)])
def test_a_step_allocates_nothing(T, topk):
    """Every buffer of the layer, its scratch memory included, is there once the layer is."""
    ex = example()
    E, k, D, Fh = 4, 2, 384, 256
    dev = torch.device("cuda")
    routed = ex.random_weights(E, 2 * Fh, D, "e4m3", dev) + ex.random_weights(E, D, Fh, "e4m3", dev)
    up, down = ex.random_weights(1, 2 * Fh, D, "int8", dev), ex.random_weights(1, D, Fh, "int8", dev)
    shared = (up[0][0], up[1][0], down[0][0], down[1][0])
    layer = ex.DecodeMoeLayer(T, routed, shared) if topk is None else ex.DecodeMoeLayer(T, routed, shared, topk)
    x = torch.randn((T, D), device=dev).bfloat16()
    idx = torch.randint(0, E, (T, k), device=dev, dtype=torch.int32)
    wt = torch.rand((T, k), device=dev).bfloat16()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    layer(x, idx, wt)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
