"""One decode step of a mixture-of-experts feed-forward layer: routed experts plus a shared expert.

The routed experts of up to 64 tokens run in ``moe_few`` (e4m3 weights with 128x128 block scales, or int8 weights with
channel scales); the shared expert, which sees every token, is an int8 feed-forward layer: ``linear_i8`` for the stacked
up-projections and ``silu_mul_linear_i8`` for the gate and the down-projection.  Nothing is synchronised and every
buffer is allocated once, so the step is captured into a HIP graph and replayed.

    python examples/decode_moe_layer.py --tokens 16 [--routed int8] [--experts 256 --topk 8 --dim 7168 --inter 2048]

prints the step's time, eager and as a graph, and how far a token's output is from a plain fp32 computation.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_act_amd as ds  # noqa: E402


class DecodeMoeLayer:
    """The layer's weights and, for a fixed number of tokens, its buffers.

    ``routed = (w13, w13_s, w2, w2_s)`` as ``moe_few`` takes them; ``shared`` is one int8 expert: ``w13 [2F, D]``,
    ``w13_s [2F]``, ``w2 [D, F]``, ``w2_s [D]``.  ``topk``: the most experts a token is routed to."""

    def __init__(self, tokens, routed, shared, topk=16):
        self.routed, self.shared = routed, shared
        D, device = routed[0].shape[2], routed[0].device
        F2, F = shared[0].shape[0], shared[2].shape[1]
        self.gate_up = torch.empty((tokens, F2), dtype=torch.bfloat16, device=device)
        self.y = torch.empty((tokens, D), dtype=torch.bfloat16, device=device)
        self.out = torch.empty((tokens, D), dtype=torch.bfloat16, device=device)
        # scratch memory of the three calls, which follow each other on one stream
        need = max(ds.moe_few_workspace_bytes(tokens, topk, routed[2].shape[2]),
                   ds.linear_i8_workspace_bytes(tokens, F2, D), ds.linear_i8_workspace_bytes(tokens, D, F, gated=True))
        self.work = torch.empty(need, dtype=torch.uint8, device=device)

    def __call__(self, x, indices, weights):
        """bf16 ``[tokens, D]`` for bf16 ``x [tokens, D]``, int32 ``indices`` and bf16 ``weights [tokens, k]``."""
        w13, w13_s, w2, w2_s = self.shared
        F = w2.shape[1]
        ds.moe_few(x, *self.routed, indices, weights, out=self.out, workspace=self.work)
        ds.linear_i8(x, w13, w13_s, out=self.gate_up, workspace=self.work)
        ds.silu_mul_linear_i8(self.gate_up[:, :F], self.gate_up[:, F:], w2, w2_s, out=self.y, workspace=self.work)
        return self.out.add_(self.y)


def random_weights(E, N, K, fmt, device):
    """(codes, scales) of E random matrices [N, K] with entries of about 1 / sqrt(K)."""
    if fmt == "int8":
        q = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device=device)
        return q, torch.full((E, N), 1.0 / (73.0 * K ** 0.5), device=device)
    # random bytes without the two NaNs: every finite e4m3 value is equally likely, root mean square about 113
    q = torch.randint(0, 127, (E, N, K), dtype=torch.uint8, device=device)
    q |= torch.randint(0, 2, (E, N, K), dtype=torch.uint8, device=device) << 7
    return q, torch.full((E, ds.kblocks(N), ds.kblocks(K)), 1.0 / (113.0 * K ** 0.5), device=device)


def real(q, s):
    """A stored weight [N, K] as fp32."""
    if q.dtype == torch.int8:
        return q.float() * s[:, None]
    v = q.view(torch.float8_e4m3fn).float()
    return v * s.repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]


def plain(layer, x, indices, weights, t):
    """Token t's output in fp32, without quantised activations."""
    def expert(w13, s13, w2, s2):
        g, u = (real(w13, s13) @ x[t].float()).chunk(2)
        return real(w2, s2) @ (torch.nn.functional.silu(g) * u)

    y = expert(*layer.shared)
    for e, w in zip(indices[t].tolist(), weights[t].tolist()):
        y += w * expert(*(v[e] for v in layer.routed))
    return y


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
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--experts", type=int, default=256)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--dim", type=int, default=7168)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--routed", choices=["e4m3", "int8"], default="e4m3")
    a = ap.parse_args()
    torch.manual_seed(0)
    dev = torch.device("cuda")
    routed = random_weights(a.experts, 2 * a.inter, a.dim, a.routed, dev) + \
        random_weights(a.experts, a.dim, a.inter, a.routed, dev)
    up, down = random_weights(1, 2 * a.inter, a.dim, "int8", dev), random_weights(1, a.dim, a.inter, "int8", dev)
    layer = DecodeMoeLayer(a.tokens, routed, (up[0][0], up[1][0], down[0][0], down[1][0]), a.topk)
    x = torch.randn((a.tokens, a.dim), device=dev).bfloat16()
    score, indices = torch.randn((a.tokens, a.experts), device=dev).sigmoid().topk(a.topk)
    weights, indices = (score / score.sum(1, keepdim=True)).bfloat16(), indices.int()

    want = plain(layer, x, indices, weights, a.tokens - 1)
    got = layer(x, indices, weights)[a.tokens - 1].float()
    error = float((got - want).norm() / want.norm())
    eager = microseconds(lambda: layer(x, indices, weights))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, indices, weights)
    replay = microseconds(graph.replay)
    print(f"{a.tokens} tokens, {indices.unique().numel()} of {a.experts} {a.routed} experts hit: eager {eager:.1f} us, "
          f"graph {replay:.1f} us a step; relative error against fp32 {error:.4f}")


if __name__ == "__main__":
    main()
