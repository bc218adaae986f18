"""Measured cases of the few-token expert layer and the 8-bit integer linear layer.

Three operators, each in its plain form (elementary torch operations in fp32,
rounded once at the end) and through the library's entry points:

* ``linear``: bf16 rows quantised to int8 with one scale per row (token), times
  an int8 weight [N, K] with one scale per output channel, to bf16;
* ``gated``: the same product of SiLU(g) * u (the down-projection of a gated
  feed-forward layer), the gate evaluated on the way into the quantiser;
* ``moe``: a whole routed-expert layer for a few tokens, from the gate's expert
  indices and weights to the combined output, with e4m3 weights in 128x128
  scale blocks or int8 weights with a scale per output channel.
"""

import math

import numpy as np
import torch

own = False

AMAX_FLOOR = 2.0 ** -100        # least row maximum the quantiser divides by
BLOCK = 128


def listed():
    return [
        # one generated token through the query down-projection: launch latency and an 11 MB weight
        dict(name="linear one row", op="linear", M=1, N=1536, K=7168),
        # the same projection for a decode batch of 32 sequences
        dict(name="linear decode batch", op="linear", M=32, N=1536, K=7168),
        # sizes that divide nothing: a ragged batch, rows only 8-byte aligned
        dict(name="linear ragged", op="linear", M=333, N=2500, K=1000),
        # prefill of 4096 tokens through one up-projection of the dense feed-forward layer
        dict(name="linear prefill", op="linear", M=4096, N=18432, K=7168),
        # down-projection of the shared expert for a decode batch
        dict(name="gated decode batch", op="gated", M=64, N=7168, K=2048),
        # down-projection of the dense feed-forward layer in prefill
        dict(name="gated prefill", op="gated", M=4096, N=7168, K=18432),
        # one generated token: 8 experts of 256, every expert with one row
        dict(name="moe one token", op="moe", T=1, E=256, G=256, k=8, D=7168, F=2048, fmt="e4m3"),
        # a small decode batch: about 70 distinct experts, one to a few rows each
        dict(name="moe 16 tokens", op="moe", T=16, E=256, G=256, k=8, D=7168, F=2048, fmt="e4m3"),
        # one rank of 8-way expert parallelism: 32 of 256 experts, most choices belong to other ranks
        dict(name="moe rank of 8, 64 tokens", op="moe", T=64, E=32, G=256, k=8, D=7168, F=2048, fmt="e4m3"),
        # int8 expert weights, 4 tokens
        dict(name="moe int8", op="moe", T=4, E=64, G=64, k=8, D=7168, F=2048, fmt="int8"),
        # a small layer of sizes that divide nothing, where latency counts
        dict(name="moe small odd", op="moe", T=5, E=8, G=8, k=2, D=1000, F=714, fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks(rng, lo, hi, block):
    """A size of whole blocks, as most layers have; 24 blocks of 128 are left out (no layer here has them)."""
    n = (_log(rng, lo, hi) + block - 1) // block * block
    return n + block if n == 24 * BLOCK else n


def draw(rng):
    if rng.random() < 0.5:
        op = rng.choice(["linear", "gated"])
        M = _log(rng, 1, 4096)
        if rng.random() < 0.6:
            N, K = _blocks(rng, 256, 18000, 64), _blocks(rng, 256, 18000, 128)
        else:
            N, K = (2 * _log(rng, 128, 9000) + 1 for _ in range(2))
        if M == 24 * BLOCK:
            M += 1
        while M * N * K > 4096 * 18432 * 7168:
            M = max(1, M // 2)
        return dict(op=op, M=M, N=N, K=K)
    T = _log(rng, 1, 64)
    G = rng.choice([8, 16, 32, 64, 128, 256])
    E = G if rng.random() < 0.6 else max(2, G // rng.choice([2, 4, 8]))
    k = rng.randint(1, min(8, G))
    if rng.random() < 0.6:
        D, F = _blocks(rng, 256, 7000, 128), _blocks(rng, 128, 2000, 128)
    else:
        D, F = 2 * _log(rng, 128, 3500) + 1, _log(rng, 100, 2000)
    return dict(op="moe", T=T, E=E, G=G, k=k, D=D, F=F, fmt=rng.choice(["e4m3", "int8"]))


# ---- inputs --------------------------------------------------------------------------------


def _kb(n):
    return (n + BLOCK - 1) // BLOCK


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _routing(case, seed):
    """The gate's choice on the host: k distinct experts of G per token with Zipf(1.1) popularity
    (the skew of the repository's routed workload), as indices relative to the rank's first expert
    (entries outside [0, E) belong to other ranks), and positive weights that sum to 2.5."""
    g = _gen(seed, "cpu")
    T, G, E, k = case["T"], case["G"], case["E"], case["k"]
    logp = torch.empty(G, dtype=torch.float64)
    logp[torch.randperm(G, generator=g)] = -1.1 * torch.log(torch.arange(1, G + 1, dtype=torch.float64))
    u = torch.rand((T, G), generator=g, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)
    idx = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    first = int(torch.randint(0, G // E, (1,), generator=g)) * E
    w = 0.05 + 0.95 * torch.rand((T, k), generator=g)
    w = 2.5 * w / w.sum(1, keepdim=True)
    return (idx - first).to(torch.int32), w.to(torch.bfloat16)


def _weight(shape, fmt, g, device):
    """Weights of N(0, 0.02): the stored codes and their scales (block maxima near 448, channel maxima
    near 127), drawn directly in the stored format."""
    *lead, n, k = shape
    if fmt == "int8":
        q = torch.empty(shape, dtype=torch.int8, device=device)
        s = (0.02 / 32) * (0.8 + 0.4 * torch.rand((*lead, n), generator=g, device=device))
    else:
        q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=device)
        s = (0.02 / 110) * (0.8 + 0.4 * torch.rand((*lead, _kb(n), _kb(k)), generator=g, device=device))
    flat = q.view(-1, k)
    step = max(1, (1 << 28) // k)
    for r in range(0, flat.shape[0], step):
        part = flat[r:r + step]
        v = torch.randn(part.shape, generator=g, device=device)
        part.copy_(v.mul_(32).round_().clamp_(-127, 127) if fmt == "int8" else v.mul_(110).clamp_(-448, 448))
    return q, s


def _activations(M, K, g, device, outliers=False):
    x = torch.randn((M, K), generator=g, device=device)
    if outliers:                    # 1% of the channels 20 times larger, as activations have them
        x *= 1 + 19 * (torch.rand((K,), generator=g, device=device) < 0.01).float()
    return x.to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    st = dict(case)
    if case["op"] == "moe":
        E, D, F = case["E"], case["D"], case["F"]
        st["x"] = _activations(case["T"], D, g, dev)
        st["w13"], st["s13"] = _weight((E, 2 * F, D), case["fmt"], g, dev)
        st["w2"], st["s2"] = _weight((E, D, F), case["fmt"], g, dev)
        idx, w = _routing(case, seed)
        st["idx"], st["wt"] = idx.to(dev), w.to(dev)
        return st
    st["w"], st["ws"] = _weight((case["N"], case["K"]), "int8", g, dev)
    st["x"] = _activations(case["M"], case["K"], g, dev, outliers=case["op"] == "linear")
    if case["op"] == "gated":
        st["u"] = _activations(case["M"], case["K"], g, dev)
    return st


# ---- the plain forms -----------------------------------------------------------------------


def _plain_linear(x, w, ws):
    amax = x.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
    top = torch.full_like(amax, 127.0)
    q = torch.round(x * (top / amax))
    return ((q @ w.float().t()) * ((amax / top) * ws)).to(torch.bfloat16)


def _plain_weight(q, s):
    """fp32 values of stacked weights [..., n, k]."""
    w = q.float()
    if q.dtype == torch.int8:
        return w.mul_(s.unsqueeze(-1))
    rows = torch.arange(w.shape[-2], device=w.device) // BLOCK
    cols = torch.arange(w.shape[-1], device=w.device) // BLOCK
    return w.mul_(s[..., rows, :][..., cols])


def _take(q, e):
    return q.view(torch.uint8)[e].view(q.dtype)


def _plain_moe(st):
    x, idx, wt = st["x"].float(), st["idx"].long(), st["wt"].float()
    T, k = idx.shape
    E, F = st["E"], st["F"]
    here = (idx >= 0) & (idx < E)
    if T * k < E:
        # every pair's expert on its own
        e = torch.where(here, idx, torch.zeros_like(idx)).reshape(-1)
        xs = x.repeat_interleave(k, 0).unsqueeze(-1)
        gu = (_plain_weight(_take(st["w13"], e), st["s13"][e]) @ xs).squeeze(-1)
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        y = (_plain_weight(_take(st["w2"], e), st["s2"][e]) @ h.unsqueeze(-1)).view(T, k, -1)
        y = torch.where(here.unsqueeze(-1), y * wt.unsqueeze(-1), torch.zeros_like(y))
        return y.sum(1).to(torch.bfloat16)
    # more pairs than experts: every token through every expert, weighted by its choice
    hit = (idx.unsqueeze(-1) == torch.arange(E, device=x.device)).float()       # [T, k, E]
    share = (hit * wt.unsqueeze(-1)).sum(1).t()                                  # [E, T]
    gu = torch.matmul(_plain_weight(st["w13"], st["s13"]), x.t())               # [E, 2F, T]
    h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
    y = torch.matmul(_plain_weight(st["w2"], st["s2"]), h * share.unsqueeze(1))  # [E, D, T]
    return y.sum(0).t().contiguous().to(torch.bfloat16)


def run(st):
    if own:
        import block_scaled_fp8_act_amd as ds
        if st["op"] == "linear":
            return ds.linear_i8(st["x"], st["w"], st["ws"])
        if st["op"] == "gated":
            return ds.silu_mul_linear_i8(st["x"], st["u"], st["w"], st["ws"])
        return ds.moe_few(st["x"], st["w13"], st["s13"], st["w2"], st["s2"], st["idx"], st["wt"])
    if st["op"] == "linear":
        return _plain_linear(st["x"].float(), st["w"], st["ws"])
    if st["op"] == "gated":
        g = st["x"].float()
        return _plain_linear(g * torch.sigmoid(g) * st["u"].float(), st["w"], st["ws"])
    return _plain_moe(st)


# ---- work and the exact results ---------------------------------------------------------------


def work(case):
    if case["op"] != "moe":
        M, N, K = case["M"], case["N"], case["K"]
        reads = (2 if case["op"] == "gated" else 1) * 2 * M * K + N * K + 4 * N
        return {"bytes": reads + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))
    experts = pairs = 0
    for seed in range(4):           # the routing's mean over a few draws
        idx = _routing(case, seed)[0]
        mine = idx[(idx >= 0) & (idx < E)]
        experts += mine.unique().numel() / 4
        pairs += mine.numel() / 4
    scales = (2 * F + D) if case["fmt"] == "int8" else _kb(2 * F) * _kb(D) + _kb(D) * _kb(F)
    return {"bytes": int(experts * (3 * D * F + 4 * scales) + 4 * T * D + 6 * T * k), "flops": int(pairs * 6 * D * F)}


def _e4m3_values(device):
    """The 256 values of the format: bias 7, subnormal steps of 2^-9, S.1111.111 is NaN."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = math.nan if e == 15 and m == 7 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        v.append(-a if c & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=device)


def _exact_weight(q, s):
    if q.dtype == torch.int8:
        return q.double() * s.double()[:, None]
    w = _e4m3_values(q.device)[q.view(torch.uint8).long()]
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= float(s[i, j])
    return w


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "moe":
        x, idx, wt = st["x"].double(), st["idx"].cpu().numpy(), st["wt"].double()
        F = case["F"]
        out = torch.zeros_like(x)
        s13, s2 = st["s13"], st["s2"]
        if case["fmt"] != "int8":
            s13, s2 = s13.cpu(), s2.cpu()
        for e in range(case["E"]):
            t, j = (torch.from_numpy(v).to(x.device) for v in np.nonzero(idx == e))
            if t.numel() == 0:
                continue
            gu = x[t] @ _exact_weight(st["w13"][e], s13[e]).t()
            g, u = gu[:, :F], gu[:, F:]
            y = (g / (1 + torch.exp(-g)) * u) @ _exact_weight(st["w2"][e], s2[e]).t()
            out.index_add_(0, t, y * wt[t, j][:, None])
        return out
    x = st["x"].double()
    if case["op"] == "gated":
        x = x / (1 + torch.exp(-x)) * st["u"].double()
    # the quantiser's steps are fp32 operations, each correctly rounded, by definition
    xs = x.float().cpu().numpy()
    amax = np.maximum(np.abs(xs).max(axis=1, keepdims=True), np.float32(AMAX_FLOOR))
    q = np.rint(xs * (np.float32(127) / amax)).astype(np.float64)
    s = (amax / np.float32(127)).astype(np.float64)
    acc = torch.from_numpy(q).to(x.device) @ st["w"].double().t()       # whole numbers below 2^53
    return acc * torch.from_numpy(s).to(x.device) * st["ws"].double()
