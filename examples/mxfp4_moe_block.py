"""A mixture-of-experts feed-forward block with MXFP4 weights and activations: norm, gate, routed experts, residual.

The block takes the previous block's output and the residual stream; one call adds the two, norms the sum and quantises
it (``add_rms_norm``).  The router's product, the choice of experts (``moe_gate``) and the rows' order (``moe_route``)
follow, then the experts: the up-projection of the tokens' rows, read through the routing's index
(``grouped_gemm_mxfp4``), the gate and the next quantisation (``silu_mul_mxfp4_quant``), the down-projection and the
weighted sum (``moe_combine``).  Nothing is synchronised, so the block is captured into a HIP graph and replayed.

The router is an MXFP4 weight here, since the norm hands its result out in that format alone, and its logits are bf16.
The choice of experts hangs on them: a model trained with its router in bf16 or fp32 keeps it so, takes the router's input
from the residual stream through a norm of its own, and gives ``moe_gate`` fp32 logits.

    python examples/mxfp4_moe_block.py --tokens 64 [--experts 64 --topk 6 --groups 8 --top-groups 3 --dim 2048 --inter 1024]

prints the block's time, eager and as a graph.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_act_amd as ds  # noqa: E402


class Mxfp4MoeBlock:
    """The block's weights.  ``norm`` [D] and ``post_norm`` [D] or None; ``router``, ``w13`` and ``w2`` are MXFP4 pairs
    (codes, scales) of ``[E, D]``, ``[E, 2F, D]`` (w1 over w3) and ``[E, D, F]``; ``bias`` fp32 ``[E]`` or None."""

    def __init__(self, norm, post_norm, router, bias, w13, w2, topk, groups=1, top_groups=1, scale=1.0):
        self.norm, self.post_norm, self.router, self.bias, self.w13, self.w2 = norm, post_norm, router, bias, w13, w2
        self.topk, self.groups, self.top_groups, self.scale = topk, groups, top_groups, scale

    def __call__(self, x, stream):
        """The block's output, bf16 ``[T, D]``, for the previous block's output ``x``; ``stream`` is updated in place."""
        self.q, self.s, _ = ds.add_rms_norm(x, self.norm, residual=stream, post_weight=self.post_norm, quant="mxfp4",
                                            out=(*ds.mxfp4_empty(*x.shape, x.device), stream))
        self.logits = ds.gemm_mxfp4(self.q, self.s, *self.router)
        self.indices, self.weights = ds.moe_gate(self.logits, self.topk, bias=self.bias, groups=self.groups,
                                                 top_groups=self.top_groups, scale=self.scale)
        self.offsets, rows, token_rows = ds.moe_route(self.indices, self.w13[0].shape[0])
        self.gate_up = ds.grouped_gemm_mxfp4(self.q, self.s, *self.w13, self.offsets, rows=rows)
        F = self.gate_up.shape[1] // 2
        self.h, self.h_s = ds.silu_mul_mxfp4_quant(self.gate_up[:, :F], self.gate_up[:, F:])
        self.y = ds.grouped_gemm_mxfp4(self.h, self.h_s, *self.w2, self.offsets)
        self.rows, self.token_rows = rows, token_rows
        return ds.moe_combine(self.y, self.indices, self.weights, token_rows)


def quantised(w):
    """MXFP4 pair of a real weight [..., N, K]."""
    *lead, N, K = w.shape
    q, s = ds.mxfp4_empty(N, K, w.device, lead=tuple(lead))
    for i in range(max(1, w.numel() // (N * K))):
        ds.mxfp4_quant(w.view(-1, N, K)[i], out=(q.view(-1, *q.shape[-2:])[i], s.flatten(0, -3)[i] if lead else s))
    return q, s


def microseconds(step, n=50):
    step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        step()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--top-groups", type=int, default=3)
    ap.add_argument("--dim", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    a = ap.parse_args()
    torch.manual_seed(0)
    dev = torch.device("cuda")

    def weight(*shape):
        return quantised(torch.randn(shape, device=dev) / shape[-1] ** 0.5)
    ones = torch.ones(a.dim, dtype=torch.bfloat16, device=dev)
    block = Mxfp4MoeBlock(ones, ones, weight(a.experts, a.dim), 0.1 * torch.randn(a.experts, device=dev),
                          weight(a.experts, 2 * a.inter, a.dim), weight(a.experts, a.dim, a.inter), a.topk, a.groups,
                          a.top_groups, scale=2.5)
    x, stream = (torch.randn((a.tokens, a.dim), device=dev).bfloat16() for _ in range(2))
    eager = microseconds(lambda: block(x, stream))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, stream)
    replay = microseconds(graph.replay)
    hit = int((block.offsets.diff() > 0).sum())
    print(f"{a.tokens} tokens, {hit} of {a.experts} experts hit: eager {eager:.1f} us, graph {replay:.1f} us a block")


if __name__ == "__main__":
    main()
