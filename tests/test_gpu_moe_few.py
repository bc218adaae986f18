"""GPU checks of the few-token expert layer against the fp64 oracle, element by
element within the bound that oracle/moe_few.py derives."""

import functools

import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as ds
from block_scaled_fp8_act_amd import inputs as I
from oracle import int8 as Q8
from oracle import moe_few as MF
from oracle import quant as Q

from gpu_helpers import bf16_to_f64, dev_bf16, host_bits16

pytestmark = pytest.mark.gpu

CID = 90


@functools.lru_cache(maxsize=8)
def weights(E, D, Fh, fmt):
    quant = Q8.row_quant if fmt == "int8" else Q.weight_quant
    q13 = [quant(I.weights_f32((2 * Fh, D), CID, 2 * e, std=1.0 / max(D, 1) ** 0.5)) for e in range(E)]
    q2 = [quant(I.weights_f32((D, Fh), CID, 2 * e + 1, std=1.0 / max(Fh, 1) ** 0.5)) for e in range(E)]
    return tuple(np.stack(v) for v in zip(*q13)) + tuple(np.stack(v) for v in zip(*q2))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def routing(T, E, k, seed, G=None):
    """k distinct experts of G per token, relative to the middle of the range when G > E."""
    G = G or E
    g = I.rng(CID, 1000 + seed)
    idx = np.stack([g.permutation(G)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    w = I.to_bf16_bits(g.uniform(0.05, 1.0, (T, k)).astype(np.float32))
    return idx - (G - E) // 2, w


def run(x, ws, idx, wb, **kw):
    return ds.moe_few(dev_bf16(x), *(dev(v) for v in ws), dev(idx), dev_bf16(wb), **kw)


def check(got, x, ws, idx, wb, what=""):
    ref, bound = MF.layer(x, *ws, idx, wb)
    err = np.abs(bf16_to_f64(host_bits16(got)) - ref)
    assert np.all(err <= bound), f"{what}: {float((err / bound).max()):.3f} of the bound"
    none = ~((idx >= 0) & (idx < ws[0].shape[0])).any(axis=1)
    assert not host_bits16(got)[none].any(), "a token without experts here gets zeros"


# T, E, k, D, F: one token; columns over one, two, three and four tiles of 16; sizes around blocks of 128 and tiles of
# 32 and 16; more slots than the waves of a workgroup; a single element
CASES = [(1, 1, 1, 128, 128), (1, 8, 2, 512, 256), (1, 4, 3, 1, 1), (2, 3, 3, 17, 9), (5, 8, 2, 1000, 714),
         (16, 4, 2, 256, 128), (17, 4, 4, 256, 130), (33, 2, 2, 300, 100), (48, 3, 2, 129, 127), (64, 2, 1, 384, 160),
         (64, 32, 8, 640, 256), (7, 40, 16, 257, 65), (64, 16, 16, 128, 32), (3, 6, 2, 2304, 1024), (20, 9, 3, 130, 383)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,E,k,D,Fh", CASES)
def test_layer(T, E, k, D, Fh, fmt):
    ws = weights(E, D, Fh, fmt)
    x = I.activations((T, D), CID, 500 + T)
    idx, wb = routing(T, E, k, T)
    out = run(x, ws, idx, wb)
    check(out, x, ws, idx, wb)
    assert torch.equal(out, run(x, ws, idx, wb)), "repeated calls give the same bytes"


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,E,G,k", [(1, 4, 32, 8), (40, 4, 32, 2), (64, 2, 64, 8)])
def test_experts_of_other_ranks(T, E, G, k, fmt):
    """Indices on both sides of [0, E), tokens with no expert here among them, and the extremes of int32."""
    ws = weights(4, 384, 160, fmt)
    ws = tuple(v[:E] for v in ws)
    x = I.activations((T, 384), CID, 600 + T)
    idx, wb = routing(T, E, k, 10 + T, G)
    idx[0, 0] = np.iinfo(np.int32).min
    idx[-1, -1] = np.iinfo(np.int32).max
    if T > 1:
        idx[T // 2] = E
    check(run(x, ws, idx, wb), x, ws, idx, wb)


def test_no_expert_at_all():
    ws = weights(4, 384, 160, "e4m3")
    x = I.activations((9, 384), CID, 3)
    out = torch.full((9, 384), float("nan"), dtype=torch.bfloat16, device="cuda")
    run(x, ws, np.full((9, 2), -1, np.int32), np.full((9, 2), 0x3f80, np.uint16), out=out)
    assert not host_bits16(out).any()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_one_expert_named_twice(fmt):
    ws = weights(4, 384, 160, fmt)
    T = 18
    x = I.activations((T, 384), CID, 4)
    idx, wb = routing(T, 4, 4, 5)
    idx[:, 2] = idx[:, 0]
    idx[3] = 1
    check(run(x, ws, idx, wb), x, ws, idx, wb)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_token_depends_on_itself_alone(fmt):
    """NaN and infinities in one token, and NaN weights of experts nobody chose, touch nothing else."""
    T, E, D, Fh = 20, 6, 300, 100
    ws = [v.copy() for v in weights(E, D, Fh, fmt)]
    x = I.activations((T, D), CID, 7)
    idx, wb = routing(T, E - 1, 2, 6)
    good = run(x, ws, idx, wb)
    x[4, 10], x[11, 0] = 0x7fc0, 0xff80
    ws[1][E - 1], ws[3][E - 1] = np.nan, np.nan
    bad = run(x, ws, idx, wb)
    keep = [t for t in range(T) if t not in (4, 11)]
    assert torch.equal(bad[keep], good[keep])
    assert not bool(torch.isfinite(bad[4]).any()) and not bool(torch.isfinite(bad[11]).any())


def test_large_gate_values():
    """g far in both tails: SiLU gives g, or zero without NaN."""
    T, E, D, Fh = 4, 2, 128, 64
    ws = weights(E, D, Fh, "int8")
    x = I.activations((T, D), CID, 8, std=200.0)
    idx, wb = routing(T, E, 1, 7)
    check(run(x, ws, idx, wb), x, ws, idx, wb)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_strides_and_alignment(fmt):
    """Rows at odd addresses everywhere, an output inside a wider buffer, strided indices and weights."""
    T, E, k, D, Fh = 19, 5, 3, 333, 150
    ws = weights(E, D, Fh, fmt)
    x = I.activations((T, D), CID, 9)
    idx, wb = routing(T, E, k, 8)

    def place(a, ld, off):
        a = np.asarray(a)
        buf = torch.zeros(off + int(np.prod(a.shape[:-1])) * ld + 32, dtype=torch.from_numpy(a[:0].copy()).dtype,
                          device="cuda")
        v = buf[off:off + int(np.prod(a.shape[:-1])) * ld].view(*a.shape[:-1], ld)[..., :a.shape[-1]]
        v.copy_(dev(a))
        return v

    xb = place(x.view(np.int16), D + 3, 1).view(torch.bfloat16)
    wide = torch.full((T, D + 7), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 1:1 + D]
    got = ds.moe_few(xb, place(ws[0], D + 5, 3), place(ws[1], ws[1].shape[-1] + 2, 1), place(ws[2], Fh + 1, 7),
                     place(ws[3], ws[3].shape[-1] + 1, 1), place(idx, k + 2, 1),
                     place(wb.view(np.int16), k + 1, 1).view(torch.bfloat16), out=out)
    check(got, x, ws, idx, wb)
    assert bool((wide[:, 0] == 3.0).all()) and bool((wide[:, 1 + D:] == 3.0).all())


def test_expert_past_4_gib():
    """The last of 150 experts, whose weights lie past 4 GiB; only it is read."""
    E, D, Fh = 150, 7168, 2048
    w13 = torch.empty((E, 2 * Fh, D), dtype=torch.uint8, device="cuda")
    w2 = torch.empty((E, D, Fh), dtype=torch.uint8, device="cuda")
    s13 = torch.full((E, 2 * Fh // 128, D // 128), float("nan"), device="cuda")
    s2 = torch.full((E, D // 128, Fh // 128), float("nan"), device="cuda")
    one = weights(1, D, Fh, "e4m3")
    for t, v in zip((w13, s13, w2, s2), one):
        t[E - 1] = dev(v[0])
    x = I.activations((2, D), CID, 11)
    wb = np.full((2, 1), 0x3f80, np.uint16)
    got = ds.moe_few(dev_bf16(x), w13, s13, w2, s2, torch.full((2, 1), E - 1, dtype=torch.int32, device="cuda"),
                     dev_bf16(wb))
    check(got, x, one, np.zeros((2, 1), np.int32), wb)


def test_empty_sizes():
    ws = weights(2, 128, 64, "e4m3")
    idx, wb = routing(0, 2, 2, 1)
    assert run(np.zeros((0, 128), np.uint16), ws, idx, wb).shape == (0, 128)
    idx, wb = routing(3, 2, 2, 1)
    E, D = 2, 128
    none = (np.zeros((E, 0, D), np.uint8), np.zeros((E, 0, 1), np.float32), np.zeros((E, D, 0), np.uint8),
            np.zeros((E, 1, 0), np.float32))
    out = torch.full((3, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    run(I.activations((3, D), CID, 1), none, idx, wb, out=out)
    assert not host_bits16(out).any()


def test_near_the_grouped_pipeline():
    """The same layer through the grouped products, which quantise activations to e4m3 (3 bits of fraction: up to
    2^-4 per element, about 2.6% of random vectors; two of them, and the bf16 roundings of the pipeline)."""
    T, E, k, D, Fh = 24, 8, 2, 512, 256
    ws = weights(E, D, Fh, "e4m3")
    x = I.activations((T, D), CID, 12)
    idx, wb = routing(T, E, k, 9)
    w13, s13, w2, s2 = (dev(v) for v in ws)
    offsets, row_token, token_rows = ds.moe_route(dev(idx), E)
    a, a_s = ds.act_quant(dev_bf16(x))
    y, s = ds.grouped_gemm_silu_mul_act_quant(a, a_s, w13, s13, offsets, rows=row_token)
    pipe = ds.moe_combine(ds.grouped_gemm(y, s, w2, s2, offsets), dev(idx), dev_bf16(wb), token_rows).float()
    few = run(x, ws, idx, wb).float()
    assert float((few - pipe).norm() / pipe.norm()) < 0.08


def test_stream_and_graph():
    T, E, k, D, Fh = 6, 8, 2, 512, 256
    ws = [dev(v) for v in weights(E, D, Fh, "e4m3")]
    x = dev_bf16(I.activations((T, D), CID, 13))
    idx, wb = routing(T, E, k, 10)
    idx, wb = dev(idx), dev_bf16(wb)
    out = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    want = ds.moe_few(x, *ws, idx, wb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ds.moe_few(x, *ws, idx, wb, out=out, workspace=work)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.moe_few(x, *ws, idx, wb, out=out, workspace=work)
    for i in range(4):
        ni, nw = routing(T, E, k, 20 + i)
        x.copy_(dev_bf16(I.activations((T, D), CID, 40 + i)))
        idx.copy_(dev(ni))
        wb.copy_(dev_bf16(nw))
        work.random_()                               # nothing in it survives from one call to the next
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ds.moe_few(x, *ws, idx, wb))


def test_refusals():
    E, D, Fh, T, k = 2, 128, 64, 3, 2
    w13, s13, w2, s2 = (dev(v) for v in weights(E, D, Fh, "e4m3"))
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    wt = torch.ones((T, k), dtype=torch.bfloat16, device="cuda")
    ds.moe_few(x, w13, s13, w2, s2, idx, wt)

    def refused(*args, **kw):
        with pytest.raises(ds.Dsfp8Error):
            ds.moe_few(*args, **kw)

    refused(x.float(), w13, s13, w2, s2, idx, wt)
    refused(x, w13, s13, w2.view(torch.int8), s2, idx, wt)
    refused(x, w13.view(torch.int8), s13, w2.view(torch.int8), s2, idx, wt)      # block scales with int8 weights
    refused(x, w13[:, :-1], s13, w2, s2, idx, wt)
    refused(x, w13, s13[:, :, :0], w2, s2, idx, wt)
    refused(x, w13, s13, w2[:, :-1], s2, idx, wt)
    refused(x, w13, s13, w2, s2, idx.long(), wt)
    refused(x, w13, s13, w2, s2, idx, wt.float())
    refused(x, w13, s13, w2, s2, idx[:2], wt)
    refused(x, w13, s13, w2, s2, idx, wt, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    refused(x, w13.cpu(), s13, w2, s2, idx, wt)
    many = torch.zeros((65, D), dtype=torch.bfloat16, device="cuda")
    refused(many, w13, s13, w2, s2, torch.zeros((65, k), dtype=torch.int32, device="cuda"),
            torch.ones((65, k), dtype=torch.bfloat16, device="cuda"))
    wide = torch.zeros((T, 17), dtype=torch.int32, device="cuda")
    refused(x, w13, s13, w2, s2, wide, torch.ones((T, 17), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,E,k,D,Fh", [(3, 3, 2, 256, 144), (18, 2, 2, 512, 16), (2, 2, 1, 4224, 64),
                                        (3, 2, 1, 4112, 48), (17, 2, 2, 5008, 16), (1, 1, 1, 16, 16)])
def test_row_tiles_past_the_last_row(T, E, k, D, Fh, fmt):
    """16-byte aligned weights whose last task of 32 rows, or last workgroup of up to 32 output columns, has 16 rows
    or fewer, so that its second tile of 16 rows lies past the matrix altogether."""
    ws = weights(E, D, Fh, fmt)
    x = I.activations((T, D), CID, 700 + T)
    idx, wb = routing(T, E, k, 30 + T)
    out = run(x, ws, idx, wb)
    check(out, x, ws, idx, wb)
    assert torch.equal(out, run(x, ws, idx, wb)), "repeated calls give the same bytes"


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [6, 40])
def test_other_tokens_values_and_routing(T, fmt):
    """Token 0 of a call: the same bytes whatever the other tokens hold while all indices stay; within the bound when
    the others are routed elsewhere, nowhere, or left out, which moves the cuts of its sums."""
    E, k, D, Fh = 8, 3, 640, 384
    ws = weights(E, D, Fh, fmt)
    x = I.activations((T, D), CID, 800)
    idx, wb = routing(T, E, k, 40)
    first = run(x, ws, idx, wb)
    check(first, x, ws, idx, wb)
    other_x, other_wb = I.activations((T, D), CID, 801, std=50.0), routing(T, E, k, 41)[1]
    other_x[0], other_wb[0] = x[0], wb[0]
    assert torch.equal(run(other_x, ws, idx, other_wb)[0], first[0])
    for i in range(4):
        other = routing(T, E, k, 42 + i)[0] if i < 3 else np.full((T, k), -1, np.int32)
        other[0] = idx[0]
        check(run(x, ws, other, wb), x, ws, other, wb, f"routing {i}")
    check(run(x[:1], ws, idx[:1], wb[:1]), x[:1], ws, idx[:1], wb[:1], "alone")


def test_block_scales_inside_larger_ones():
    """Experts with a single row of block scales each, taken out of a larger grid."""
    T, E, k, D, Fh = 4, 3, 2, 128, 64
    ws = weights(E, D, Fh, "e4m3")
    x = I.activations((T, D), CID, 820)
    idx, wb = routing(T, E, k, 50)
    s13, s2 = dev(ws[1]), dev(ws[3])
    assert s13.shape == (E, 1, 1) and s2.shape == (E, 1, 1)
    grid = torch.full((E, 3, 5), float("nan"), device="cuda")
    grid[:, :1, :1], grid[:, 2:, 4:] = s13, s2
    got = ds.moe_few(dev_bf16(x), dev(ws[0]), grid[:, :1, :1], dev(ws[2]), grid[:, 2:, 4:], dev(idx), dev_bf16(wb))
    check(got, x, ws, idx, wb)
