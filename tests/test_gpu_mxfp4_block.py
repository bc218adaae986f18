"""The MXFP4 expert block: norm, router, gate, routing, experts and combine together, every step against its oracle on
what the step before it gave, then replayed as a graph."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from block_scaled_fp8_act_amd import inputs as I
from oracle import gate as GT
from oracle import int8 as Q8
from oracle import moe as M
from oracle import mxfp4 as MX
from oracle import norm as NM

from gpu_helpers import bf16_to_f64, dev_bf16, host_bits16, host_u8

pytestmark = pytest.mark.gpu

CID = 150


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_moe_block.py")
    spec = importlib.util.spec_from_file_location("mxfp4_moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def close(got, a, a_s, b, b_s, what):
    ref, bound = MX.gemm(a, a_s, b, b_s)
    err = np.abs(bf16_to_f64(got) - ref)
    assert np.all(err <= (np.abs(ref) + bound) * 2.0 ** -8 + bound), what


@pytest.mark.parametrize("T,E,k,groups,top,D,Fh,post", [(1, 8, 2, 1, 1, 256, 128, True), (7, 16, 4, 4, 2, 1000, 200, False),
                                                        (64, 32, 6, 8, 3, 544, 320, True), (300, 12, 3, 3, 2, 320, 160, True)])
def test_block(T, E, k, groups, top, D, Fh, post):
    ex = example()
    g = I.rng(CID, T)

    def weight(seed, *shape):
        w = torch.from_numpy(I.rng(CID, seed).standard_normal(shape, dtype=np.float32) / np.float32(shape[-1] ** 0.5))
        return ex.quantised(w.cuda())
    router, w13, w2 = weight(1, E, D), weight(2, E, 2 * Fh, D), weight(3, E, D, Fh)
    norm, post_norm = (torch.from_numpy((1 + 0.2 * g.standard_normal(D)).astype(np.float32)).bfloat16() for _ in range(2))
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    block = ex.Mxfp4MoeBlock(norm.cuda(), post_norm.cuda() if post else None, router, torch.from_numpy(bias).cuda(), w13, w2, k,
                             groups, top, scale=2.5)
    xb, rb = I.activations((T, D), CID, 10 + T), I.activations((T, D), CID, 11 + T)
    x, stream = dev_bf16(xb), dev_bf16(rb)
    out = block(x, stream)

    h, dh, y, dy = NM.forward(bf16_to_f64(xb), norm.double().numpy(), bf16_to_f64(rb), post_norm.double().numpy() if post else None)
    assert np.all(np.abs(bf16_to_f64(host_bits16(stream)) - h) <= dh + (np.abs(h) + dh) * 2.0 ** -8)
    q, s = host_u8(block.q), host_u8(block.s)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)[:, :D]
    a = (np.abs(y) + dy) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.maximum(1.0, a - 6))) * unit
    assert np.all(np.abs(MX.values(q, s, D) - y) <= half + dy)

    rq, rs = host_u8(router[0]), host_u8(router[1])
    close(host_bits16(block.logits), q, s, rq, rs, "router")
    idx, w = GT.gate(block.logits.float().cpu().numpy(), k, bias=bias, groups=groups, top_groups=top, scale=2.5)
    assert np.array_equal(block.indices.cpu().numpy(), idx)
    assert np.all(np.abs(bf16_to_f64(host_bits16(block.weights)) - w) <= np.abs(w) * (2.0 ** -8 + 20 * 2.0 ** -24))

    off, rows = block.offsets.cpu().numpy(), block.rows.cpu().numpy()
    gu, hq, hs, yr = host_bits16(block.gate_up), host_u8(block.h), host_u8(block.h_s), host_bits16(block.y)
    assert off[-1] == T * k
    x64 = Q8.silu_mul(gu[:, :Fh], gu[:, Fh:])
    d = (np.abs(bf16_to_f64(gu[:, :Fh])) + 8) * 2.0 ** -23
    hunit = np.repeat(np.ldexp(1.0, hs.astype(int) - 127), 32, axis=1)[:, :Fh]
    codes = MX.unpack(hq)[:, :Fh]
    assert np.all((codes == MX.encode(x64 * (1 - d) / hunit)) | (codes == MX.encode(x64 * (1 + d) / hunit)))
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        if len(r):
            close(gu[r], q[rows[r]], s[rows[r]], host_u8(w13[0][e]), host_u8(w13[1][e]), f"up {e}")
            close(yr[r], hq[r], hs[r], host_u8(w2[0][e]), host_u8(w2[1][e]), f"down {e}")
    want = M.combine(yr, host_bits16(block.weights), idx, block.token_rows.cpu().numpy())
    assert np.array_equal(host_bits16(out), want)

    # as a graph: each replay moves the residual stream on, as an eager call does
    start = stream.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block(x, stream)
    for seed in range(3):
        x.copy_(dev_bf16(I.activations((T, D), CID, 50 + seed)))
        stream.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got, moved = captured.clone(), stream.clone()
        stream.copy_(start)
        assert torch.equal(block(x, stream), got) and torch.equal(stream, moved)


def test_padding_tokens_cost_nothing():
    """Tokens whose logits are -inf go to no expert: no rows, and zeros from the combine."""
    import block_scaled_fp8_act_amd as ds
    T, E, D = 20, 8, 96
    logits = torch.randn((T, E), device="cuda")
    logits[5:9] = -float("inf")
    idx, w = ds.moe_gate(logits, 3)
    off, rows, token_rows = ds.moe_route(idx, E)
    assert int(off[-1]) == 3 * (T - 4)
    q, s = ds.mxfp4_quant(torch.randn((T, 64), device="cuda"))
    wq, ws = ds.mxfp4_quant(torch.randn((E * D, 64), device="cuda"))
    room = torch.zeros((E, D, 16), dtype=torch.uint8, device="cuda")
    room[..., :2] = ws.unflatten(0, (E, D))
    rows = torch.where(torch.arange(T * 3, device="cuda") < off[-1], rows, torch.full_like(rows, 10 ** 9))
    y = ds.grouped_gemm_mxfp4(q, s, wq.view(E, D, -1), room[..., :2], off, rows=rows)
    out = ds.moe_combine(y, idx, w, token_rows)
    assert not out[5:9].any() and torch.isfinite(out.float()).all() and out[:5].any()
