"""Measured cases of a feed-forward block's other operators: the choice of experts, the norm that
feeds a quantiser, and 4-bit microscaled (MXFP4) quantisation and products.

Each operator in its plain form (elementary torch operations in fp32, rounded once at the end) and
through the library's entry points:

* ``gate``: experts of a token from its router logits: sigmoid or softmax scores, a bias for balance,
  groups of experts, the k best, renormalised weights;
* ``round``: bf16 rows to MXFP4 (blocks of 32 along K, a power-of-two scale each, e2m1 codes) and back;
* ``linear``: bf16 rows quantised to MXFP4 times an MXFP4 weight [N, K], to bf16;
* ``gated``: the same product of SiLU(g) * u (the down-projection of a gated feed-forward layer);
* ``grouped``: MXFP4 rows, read through the routing's index, times their experts' MXFP4 weights;
* ``norm``: h = residual + scale * gate * rmsnorm(x), y = rmsnorm(h), y in bf16 or e4m3.
"""

import math

import numpy as np
import torch

own = False

MX = 32             # elements of an MXFP4 block
BLOCK = 128         # elements of an e4m3 block
EPS = 1e-6


def listed():
    return [
        # one generated token: 8 of 256 experts out of the best 4 of 8 groups; launch latency
        dict(name="gate one token", op="gate", T=1, E=256, k=8, G=8, top=4, score="sigmoid", bias=True, renorm=True,
             scale=2.5, dtype="fp32"),
        # the same choice for a long prefill
        dict(name="gate prefill", op="gate", T=16384, E=256, k=8, G=8, top=4, score="sigmoid", bias=True, renorm=True,
             scale=2.5, dtype="fp32"),
        # sizes that divide nothing: 60 experts, softmax of bf16 logits, no groups, no bias
        dict(name="gate softmax ragged", op="gate", T=777, E=60, k=4, G=1, top=1, score="softmax", bias=False,
             renorm=False, scale=1.0, dtype="bf16"),
        # rows that end inside a block of 32
        dict(name="round odd", op="round", M=333, K=1000),
        # activations of a prefill of 4096 tokens
        dict(name="round prefill", op="round", M=4096, K=7168),
        # one generated token through the query down-projection: launch latency and a 6 MB weight
        dict(name="linear one row", op="linear", M=1, N=1536, K=7168),
        # prefill of 4096 tokens through one up-projection of the dense feed-forward layer
        dict(name="linear prefill", op="linear", M=4096, N=18432, K=7168),
        # down-projection of the shared expert for a decode batch
        dict(name="gated decode batch", op="gated", M=64, N=7168, K=2048),
        # up-projection of a decode batch's routed experts: a few rows each
        dict(name="grouped decode batch", op="grouped", T=32, E=32, k=4, N=4096, K=7168),
        # the same of a prefill
        dict(name="grouped prefill", op="grouped", T=4096, E=32, k=4, N=4096, K=7168),
        # residual and norm before a block for a decode batch, e4m3 for the block-scaled products
        dict(name="norm decode batch", op="norm", T=32, D=7168, residual=True, post=False, gate="none", scale=1.0,
             out="e4m3"),
        # norms after one block and before the next, with gate and residual scale, for a prefill
        dict(name="norm sandwich prefill", op="norm", T=8192, D=7168, residual=True, post=True, gate="row", scale=0.5,
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "round", "linear", "gated", "grouped", "norm", "norm"])
    if op == "gate":
        G = rng.choice([1, 1, 2, 3, 4, 8, 16])
        E = G * max(2, _log(rng, 4, 512) // G)
        top = rng.randint(1, G)
        k = rng.randint(1, min(16, top * (E // G)))
        T = min(_log(rng, 1, 16384), 16384 * 256 // E)
        return dict(op=op, T=T, E=E, k=k, G=G, top=top, score=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.6, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    dtype=rng.choice(["fp32", "bf16"]))
    if op == "round":
        return dict(op=op, M=_log(rng, 1, 4096), K=_log(rng, 1, 7168))
    if op in ("linear", "gated"):
        M = _log(rng, 1, 4096)
        if rng.random() < 0.6:
            N, K = 64 * _log(rng, 4, 280), 128 * _log(rng, 2, 140)
        else:
            N, K = (2 * _log(rng, 128, 9000) + 1 for _ in range(2))
        while M * N * K > 4096 * 18432 * 7168:
            M = max(1, M // 2)
        return dict(op=op, M=M, N=N, K=K)
    if op == "grouped":
        E = rng.choice([4, 8, 16, 32, 64])
        k = rng.randint(1, min(8, E))
        N, K = (32 * _log(rng, 8, 128) if rng.random() < 0.6 else 2 * _log(rng, 128, 2000) + 1), 32 * _log(rng, 8, 224)
        T = _log(rng, 1, 4096)
        while T * k * N * K > 4096 * 4 * 4096 * 7168:
            T = max(1, T // 2)
        return dict(op=op, T=T, E=E, k=k, N=N, K=K)
    residual = rng.random() < 0.8
    D = 64 * _log(rng, 1, 256) if rng.random() < 0.6 else 2 * _log(rng, 32, 8000) + 1
    T = min(_log(rng, 1, 8192), 8192 * 7168 // D)
    return dict(op=op, T=T, D=D, residual=residual, post=residual and rng.random() < 0.5,
                gate=rng.choice(["none", "channel", "row"]) if residual else "none",
                scale=rng.choice([1.0, 0.5, 0.22]) if residual else 1.0, out=rng.choice(["bf16", "e4m3"]))


# ---- inputs --------------------------------------------------------------------------------


def _blocks(n, block):
    return (n + block - 1) // block


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _mx(rows, k, exponent, g, device):
    """MXFP4 matrix of normally distributed values as it is stored: codes [rows, 16 * blocks], the lower
    column of a pair in the low half of its byte, and scale bytes [rows, blocks] in rows padded to 16."""
    kb = _blocks(k, MX)
    q = torch.empty((rows, 16 * kb), dtype=torch.uint8, device=device)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=device)
    step = max(1, (1 << 27) // (MX * kb))
    for r in range(0, rows, step):
        part = q[r:r + step]
        v = torch.randn((part.shape[0], MX * kb), generator=g, device=device).mul_(2.3)
        v[:, k:] = 0
        c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        part.copy_(c[:, 0::2] | (c[:, 1::2] << 4))
    s = torch.zeros((rows, _blocks(kb, 16) * 16), dtype=torch.uint8, device=device)[:, :kb]
    s.copy_(torch.randint(exponent - 1, exponent + 2, (rows, kb), generator=g, device=device))
    return q, s


def _activations(M, K, g, device, outliers=False):
    x = torch.randn((M, K), generator=g, device=device)
    if outliers:                    # 1% of the channels 20 times larger, as activations have them
        x *= 1 + 19 * (torch.rand((K,), generator=g, device=device) < 0.01).float()
    return x.to(torch.bfloat16)


def _routing(case, seed):
    """The rows of the experts: k distinct experts of E per token with Zipf(1.1) popularity; each row's
    token and expert, by expert, and the experts' numbers of rows (on the host)."""
    g = _gen(seed, "cpu")
    T, E, k = case["T"], case["E"], case["k"]
    logp = torch.empty(E, dtype=torch.float64)
    logp[torch.randperm(E, generator=g)] = -1.1 * torch.log(torch.arange(1, E + 1, dtype=torch.float64))
    u = torch.rand((T, E), generator=g, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)
    idx = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    e, order = torch.sort(idx.flatten(), stable=True)
    return order // k, e, torch.bincount(e, minlength=E)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    st = dict(case)
    op = case["op"]
    if op == "gate":
        T, E = case["T"], case["E"]
        # every token's scores on top of the experts' popularity
        x = torch.randn((T, E), generator=g, device=dev) * 1.5 + 0.5 * torch.randn((E,), generator=g, device=dev)
        st["logits"] = x if case["dtype"] == "fp32" else x.to(torch.bfloat16)
        st["b"] = 0.1 * torch.randn((E,), generator=g, device=dev) if case["bias"] else None
    elif op == "round":
        st["x"] = _activations(case["M"], case["K"], g, dev, outliers=True)
    elif op in ("linear", "gated"):
        st["w"], st["ws"] = _mx(case["N"], case["K"], 120, g, dev)
        st["x"] = _activations(case["M"], case["K"], g, dev, outliers=op == "linear")
        if op == "gated":
            st["u"] = _activations(case["M"], case["K"], g, dev)
    elif op == "grouped":
        E, N, K = case["E"], case["N"], case["K"]
        w, ws = _mx(E * N, K, 120, g, dev)
        st["w"], st["ws"] = w.view(E, N, -1), ws.unflatten(0, (E, N))
        st["x"], st["xs"] = _mx(case["T"], K, 126, g, dev)
        rows, e, counts = _routing(case, seed)
        offsets = torch.zeros(E + 1, dtype=torch.int64)
        offsets[1:] = counts.cumsum(0)
        st["rows"], st["offsets"] = rows.to(dev, torch.int32), offsets.to(dev, torch.int32)
        # the plain form's plan: every expert's rows in `most` slots, and where each row's result is
        most = int(counts.max())
        at = torch.arange(len(rows)) - offsets[e] + e * most
        slots = torch.full((E * most,), case["T"])
        slots[at] = rows
        st["slots"], st["at"] = slots.view(E, most).to(dev), at.to(dev)
    else:
        T, D = case["T"], case["D"]
        st["x"] = _activations(T, D, g, dev, outliers=True)
        st["w"] = (1 + 0.2 * torch.randn((D,), generator=g, device=dev)).to(torch.bfloat16)
        st["r"] = _activations(T, D, g, dev) if case["residual"] else None
        st["pw"] = (1 + 0.2 * torch.randn((D,), generator=g, device=dev)).to(torch.bfloat16) if case["post"] else None
        shape = {"none": None, "channel": (D,), "row": (T, D)}[case["gate"]]
        st["g"] = torch.sigmoid(torch.randn(shape, generator=g, device=dev)).to(torch.bfloat16) if shape else None
    return st


# ---- the plain forms -----------------------------------------------------------------------


def _plain_gate(st):
    E, k, G, top = st["E"], st["k"], st["G"], st["top"]
    x = st["logits"].double()       # scores rounded once, to fp32: ties and near ties are decided on those
    if st["score"] == "sigmoid":
        score = (1 / (1 + torch.exp(-x))).float()
    else:
        p = torch.exp(x - x.amax(1, keepdim=True))
        score = (p / p.sum(1, keepdim=True)).float()
    key = score if st["b"] is None else score + st["b"]
    if G > 1:
        by = key.view(-1, G, E // G)
        if st["b"] is None:
            best = by.amax(2)
        else:
            two = torch.sort(by, dim=2, descending=True).values[:, :, :2]
            best = two.sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :top]
        mask = torch.zeros_like(best).scatter_(1, keep, 1.0)
        key = torch.where(mask.unsqueeze(2) > 0, by, torch.full_like(by, -math.inf)).view(-1, E)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, idx)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * st["scale"]).to(torch.bfloat16)


def _powers(device):
    return torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=torch.float32, device=device)


def _plain_round(x):
    """fp32 values that MXFP4 holds of fp32 rows."""
    M, K = x.shape
    kb = _blocks(K, MX)
    b = torch.nn.functional.pad(x, (0, MX * kb - K)).view(M, kb, MX)
    e = torch.frexp(b.abs().amax(2)).exponent - 3
    e = e.clamp(-127, 127).long()
    two = _powers(x.device)
    up, down = two[e + 127].unsqueeze(2), two[127 - e].unsqueeze(2)
    a = (b * down).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_max(6)
    return (torch.where(b < 0, -q, q) * up).view(M, MX * kb)[:, :K]


def _plain_values(q, s, K):
    """fp32 values [..., K] of MXFP4 codes and scale bytes."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    v = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), -1)
    v = v.view(*q.shape[:-1], s.shape[-1], MX) * _powers(q.device)[s.int()].unsqueeze(-1)
    return v.flatten(-2)[..., :K]


def _silu_mul(g, u):
    g = g.float()
    return g * torch.sigmoid(g) * u.float()


def _plain_grouped(st):
    K = st["K"]
    x = torch.nn.functional.pad(_plain_values(st["x"], st["xs"], K), (0, 0, 0, 1))     # a row of zeros behind the last
    w = _plain_values(st["w"], st["ws"], K)
    y = torch.matmul(x[st["slots"]], w.transpose(1, 2))                                # [E, most, N]
    return y.flatten(0, 1)[st["at"]].to(torch.bfloat16)


def _plain_norm(st):
    D = st["D"]
    h = st["x"].float()
    if st["post"]:
        h = h * torch.rsqrt((h * h).sum(1, keepdim=True) / D + EPS) * st["pw"].float()
    if st["g"] is not None:
        h = h * st["g"].float()
    if st["residual"]:
        h = st["r"].float() + st["scale"] * h
    y = h * torch.rsqrt((h * h).sum(1, keepdim=True) / D + EPS) * st["w"].float()
    if st["out"] == "bf16":
        out = [y.to(torch.bfloat16)]
    else:
        kb = _blocks(D, BLOCK)
        b = torch.nn.functional.pad(y, (0, BLOCK * kb - D)).view(-1, kb, BLOCK)
        s = b.abs().amax(2).clamp_min(1e-4) / torch.full((), 448.0, device=y.device)
        q = (b / s.unsqueeze(2)).clamp(-448, 448).view(-1, BLOCK * kb)[:, :D]
        out = [q.to(torch.float8_e4m3fn), s]
    return out + ([h.to(torch.bfloat16)] if st["residual"] else [])


def _own(st):
    import block_scaled_fp8_act_amd as ds
    op = st["op"]
    if op == "gate":
        return ds.moe_gate(st["logits"], st["k"], bias=st["b"], score=st["score"], groups=st["G"], top_groups=st["top"],
                           renormalize=st["renorm"], scale=st["scale"])
    if op == "round":
        q, s = ds.mxfp4_quant(st["x"])
        return ds.mxfp4_dequant(q, s, st["K"])
    if op == "linear":
        return ds.linear_mxfp4(st["x"], st["w"], st["ws"])
    if op == "gated":
        q, s = ds.silu_mul_mxfp4_quant(st["x"], st["u"])
        return ds.gemm_mxfp4(q, s, st["w"], st["ws"])
    if op == "grouped":
        return ds.grouped_gemm_mxfp4(st["x"], st["xs"], st["w"], st["ws"], st["offsets"], rows=st["rows"])
    quant = None if st["out"] == "bf16" else st["out"]
    got = ds.add_rms_norm(st["x"], st["w"], residual=st["r"], post_weight=st["pw"], gate=st["g"], scale=st["scale"],
                          eps=EPS, quant=quant)
    got = list(got) if isinstance(got, tuple) else [got]
    if quant == "e4m3":
        got[0] = got[0].view(torch.float8_e4m3fn)
    return got


def run(st):
    if own:
        return _own(st)
    op = st["op"]
    if op == "gate":
        return _plain_gate(st)
    if op == "round":
        return _plain_round(st["x"].float()).to(torch.bfloat16)
    if op == "linear":
        return (_plain_round(st["x"].float()) @ _plain_values(st["w"], st["ws"], st["K"]).t()).to(torch.bfloat16)
    if op == "gated":
        x = _plain_round(_silu_mul(st["x"], st["u"]))
        return (x @ _plain_values(st["w"], st["ws"], st["K"]).t()).to(torch.bfloat16)
    if op == "grouped":
        return _plain_grouped(st)
    return _plain_norm(st)


# ---- work and the exact results ---------------------------------------------------------------


def _mx_bytes(rows, k):
    return rows * 17 * _blocks(k, MX)


def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["dtype"] == "fp32" else 2) + (4 * E if case["bias"] else 0) + 6 * T * k,
                "flops": 4 * T * E}
    if op == "round":
        return {"bytes": 4 * case["M"] * case["K"], "flops": 4 * case["M"] * case["K"]}
    if op in ("linear", "gated"):
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (4 if op == "gated" else 2) * M * K + _mx_bytes(N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "grouped":
        N, K = case["N"], case["K"]
        T, pairs = case["T"], case["T"] * case["k"]
        # experts that some token chose, the mean over a few draws of the routing
        experts = sum(int((_routing(case, seed)[2] > 0).sum()) for seed in range(4)) / 4
        return {"bytes": int(experts * _mx_bytes(N, K)) + _mx_bytes(T, K) + pairs * (2 * N + 4), "flops": 2 * pairs * N * K}
    T, D = case["T"], case["D"]
    each = 2 + (4 if case["residual"] else 0) + (2 if case["gate"] == "row" else 0)
    y = 2 * D if case["out"] == "bf16" else D + 4 * _blocks(D, BLOCK)
    return {"bytes": T * (D * each + y) + 4 * D, "flops": 12 * T * D}


_HALVES = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]     # between the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_round(x):
    """What MXFP4 holds of 64-bit rows: the nearest magnitude, halfway cases to the even code."""
    out = torch.zeros_like(x)
    for b in range(0, x.shape[1], MX):
        v = x[:, b:b + MX]
        top = v.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.floor(torch.log2(top.clamp_min(1e-300))), torch.full_like(top, -125.0))
        e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e)) - 2
        unit = torch.exp2(e.clamp(-127, 127))
        a = (v / unit).abs()
        code = torch.zeros_like(a, dtype=torch.int64)
        for i, h in enumerate(_HALVES):
            code += ((a >= h) if i % 2 else (a > h)).long()
        out[:, b:b + MX] = torch.tensor(_E2M1, dtype=x.dtype, device=x.device)[code] * torch.sign(v) * unit
    return out


def _exact_values(q, s, K):
    q, w = q.long(), torch.zeros((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    mag = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)
    for half in range(2):
        c = (q >> (4 * half)) & 15
        w[:, half::2] = mag[c & 7] * (1 - 2 * (c >> 3))
    w *= torch.exp2(s.double() - 127).repeat_interleave(MX, 1)
    return w[:, :K]


def _exact_gate(st):
    x = st["logits"].double().cpu().numpy()
    T, E, k, G, top = (st[n] for n in ("T", "E", "k", "G", "top"))
    # the operator's scores and keys are fp32 values, each rounded once, by definition
    if st["score"] == "sigmoid":
        score = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    else:
        p = np.exp(x - x.max(axis=1, keepdims=True))
        score = p / p.sum(axis=1, keepdims=True)
    score = score.astype(np.float32)
    key = score + st["b"].cpu().numpy() if st["bias"] else score.copy()
    if G > 1:
        by = key.reshape(T, G, E // G)
        ranked = -np.sort(-by, axis=2)
        best = ranked[:, :, 0] + ranked[:, :, 1] if st["bias"] else ranked[:, :, 0]
        place = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
        key = np.where((place < top)[:, :, None], by, np.float32(-np.inf)).reshape(T, E)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(score, idx, 1).astype(np.float64)
    if st["renorm"]:
        w /= w.sum(axis=1, keepdims=True)
    return torch.from_numpy(idx.astype(np.int32)), torch.from_numpy(w * st["scale"])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(st)
    x = st["x"]
    if op == "round":
        return _exact_round(x.double())
    if op in ("linear", "gated"):
        v = x.double()
        if op == "gated":
            v = v / (1 + torch.exp(-v)) * st["u"].double()
        return _exact_round(v) @ _exact_values(st["w"], st["ws"], case["K"]).t()
    if op == "grouped":
        v = _exact_values(x, st["xs"], case["K"])
        off, rows = st["offsets"].tolist(), st["rows"].long()
        out = torch.zeros((len(rows), case["N"]), dtype=torch.float64, device=x.device)
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                r = slice(off[e], off[e + 1])
                out[r] = v[rows[r]] @ _exact_values(st["w"][e], st["ws"][e], case["K"]).t()
        return out
    h = x.double()
    if st["pw"] is not None:
        h = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * st["pw"].double()
    if st["g"] is not None:
        h = h * st["g"].double()
    if st["r"] is not None:
        h = st["r"].double() + case["scale"] * h
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * st["w"].double()
    last = [h] if st["r"] is not None else []
    if case["out"] == "bf16":
        return [y] + last
    q, s = torch.zeros_like(y), []
    for b in range(0, y.shape[1], BLOCK):
        v = y[:, b:b + BLOCK]
        s.append(v.abs().amax(1).clamp_min(1e-4) / 448)
        a = v / s[-1][:, None]
        unit = torch.exp2(torch.floor(torch.log2(a.abs().clamp_min(2.0 ** -6))) - 3)      # 8 steps a binade
        q[:, b:b + BLOCK] = (torch.round(a / unit) * unit).clamp(-448, 448)
    return [q, torch.stack(s, 1)] + last
