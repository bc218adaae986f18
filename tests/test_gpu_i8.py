"""GPU checks of the int8 row quantiser, product and linear layer.

The quantiser's steps and the product's (exact integer sums, two fp32
multiplications, one rounding to bf16) are defined operation by operation, so
codes, scales and outputs are compared bit for bit.  The gated forms evaluate
SiLU with the hardware exponential and reciprocal: relative to fp64, the
argument of the exponential is rounded once (|g| * log2(e) * 2^-24 in the
exponent) and the exponential, reciprocal and three products a few 2^-24 more,
so h is within (|g| + 8) * 2^-23 of its value; a code may then differ from the
rounded fp64 quotient by that times 127 beyond the half unit of rounding.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as ds
from block_scaled_fp8_act_amd import inputs as I
from oracle import formats as F
from oracle import int8 as Q8

from gpu_helpers import dev_bf16, host_bits16

pytestmark = pytest.mark.gpu

CID = 80    # SeedSequence word of these tests


def bits(shape, tensor, std=1.0, outliers=0.0):
    return I.activations(shape, CID, tensor, std=std, outlier_frac=outliers)


def strided(rows, cols, ld, offset, dtype):
    """A [rows, cols] view with row stride ld, starting `offset` elements into its buffer."""
    buf = torch.zeros(offset + max(rows, 1) * ld + 64, dtype=dtype, device="cuda")
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def i8(shape, tensor):
    return I.rng(CID, tensor).integers(-127, 128, shape, dtype=np.int8)


def dev_i8(a, ld=None, offset=0):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    if ld is None:
        return t
    v = strided(a.shape[0], a.shape[1], ld, offset, torch.int8)
    v.copy_(t)
    return v


ROWS = [(1, 1), (1, 7), (3, 8), (2, 129), (5, 1000), (64, 512), (33, 2048), (7, 2500), (4, 4096), (130, 7168),
        (3, 18432), (2, 40001), (1500, 384), (9, 0)]


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_quant_bit_exact(M, K, dtype):
    b = bits((M, K), 1, outliers=0.01)
    x = F.bf16_to_f32(b) if dtype == "bf16" else I.weights_f32((M, K), CID, 2)
    y, s = ds.row_quant_i8(dev_bf16(b) if dtype == "bf16" else torch.from_numpy(x).cuda())
    yr, sr = Q8.row_quant(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), sr.view(np.uint32))
    assert np.array_equal(y.cpu().numpy(), yr)


@pytest.mark.parametrize("offset,ldx,ldy,K", [(1, 1003, 1001, 1000), (3, 520, 523, 512), (8, 136, 144, 100),
                                              (5, 9001, 9003, 9000)])
def test_row_quant_strides_and_alignment(offset, ldx, ldy, K):
    M = 6
    b = bits((M, K), 3)
    x = strided(M, K, ldx, offset, torch.bfloat16)
    x.copy_(dev_bf16(b))
    y = strided(M, K, ldy, offset, torch.int8)
    whole = y.as_strided((M, ldy), (ldy, 1))
    whole.fill_(99)
    s = torch.empty(M, device="cuda")
    ds.row_quant_i8(x, out=(y, s))
    yr, sr = Q8.row_quant(F.bf16_to_f32(b))
    assert np.array_equal(y.cpu().numpy(), yr) and np.array_equal(s.cpu().numpy(), sr)
    assert bool((whole[:-1, K:] == 99).all()), "bytes between rows were written"


def test_row_quant_special_rows():
    K = 300
    x = np.zeros((9, K), np.float32)
    x[1] = 1e-38                                     # below the floor's quantum
    x[2, 5] = np.inf
    x[3, 7] = np.nan
    x[4, 0] = -np.inf
    x[5] = -0.0
    x[6, ::3] = 254.0
    x[6, 1::3] = 3.0                                 # 127 / 254 = 0.5: 1.5 rounds to 2
    x[6, 2::3] = -1.0                                # -0.5 rounds to -0
    x[7] = np.linspace(-1, 1, K)
    x[8, K - 1] = 3e38
    y, s = ds.row_quant_i8(torch.from_numpy(x).cuda())
    y, s = y.cpu().numpy(), s.cpu().numpy()
    good = [0, 1, 5, 6, 7, 8]
    yr, sr = Q8.row_quant(x[good])
    assert np.array_equal(y[good], yr) and np.array_equal(s[good], sr)
    assert s[2] == np.inf and s[4] == np.inf and np.isnan(s[3])
    # a product of such a row shows it, in that row alone
    w = torch.ones((5, K), dtype=torch.int8, device="cuda")
    c = ds.gemm_i8(torch.from_numpy(y).cuda(), torch.from_numpy(s).cuda(), w, torch.ones(5, device="cuda")).float()
    fin = torch.isfinite(c).all(1).cpu().numpy()
    assert fin.tolist() == [True, True, False, False, False, True, True, True, True]


@pytest.mark.parametrize("M,K", [(1, 1), (3, 130), (17, 2048), (5, 18432), (2, 33001), (300, 714)])
def test_silu_mul_row_quant(M, K):
    g, u = bits((M, K), 4, std=3.0), bits((M, K), 5)
    gu = torch.cat([dev_bf16(g), dev_bf16(u)], 1)    # the halves of one product
    y, s = ds.silu_mul_row_quant_i8(gu[:, :K], gu[:, K:])
    h = Q8.silu_mul(g, u)
    rel = (np.abs(F.bf16_to_f32(g).astype(np.float64)) + 8) * 2.0 ** -23
    amax = np.maximum(np.abs(h).max(1), 2.0 ** -100)
    at = np.abs(h).argmax(1)
    tol = rel.max(1)
    s64 = s.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s64 * 127 / amax - 1) <= tol + 2.0 ** -22)
    quot = h * (127 / amax)[:, None]
    assert np.all(np.abs(y.cpu().numpy() - quot) <= 0.5 + 127 * 2 * tol[:, None] + 2.0 ** -16)
    assert np.all(np.abs(y.cpu().numpy()[np.arange(M), at]) == 127)


GEMMS = [(1, 1, 1), (1, 5, 16), (1, 1536, 7168), (3, 17, 31), (16, 256, 128), (17, 300, 144), (32, 1536, 7168),
         (33, 100, 1000), (48, 513, 2048), (64, 64, 64), (65, 129, 127), (100, 2500, 1000), (128, 128, 384),
         (200, 640, 512), (333, 2500, 1000), (256, 256, 4096), (513, 1025, 272), (1000, 2304, 896),
         (2048, 2048, 256), (1300, 4000, 1040), (5, 18432, 512), (300, 1, 77), (0, 8, 8), (8, 0, 8), (9, 9, 0)]


@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_bit_exact(M, N, K):
    a, b = i8((M, K), 10), i8((N, K), 11)
    g = I.rng(CID, 12)
    a_s, b_s = (g.uniform(0.5, 2.0, n).astype(np.float32) * np.float32(0.01) for n in (M, N))
    c = torch.full((M, N), -1.0, dtype=torch.bfloat16, device="cuda")
    ds.gemm_i8(dev_i8(a), torch.from_numpy(a_s).cuda(), dev_i8(b), torch.from_numpy(b_s).cuda(), out=c)
    assert np.array_equal(host_bits16(c), Q8.gemm(a, a_s, b, b_s))


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (20, 96, 500), (70, 260, 600), (600, 700, 1024), (2000, 1100, 513)])
@pytest.mark.parametrize("how", ["odd", "wide", "offset16"])
def test_gemm_strides_and_alignment(M, N, K, how):
    """Rows at odd addresses, wide 16-byte aligned rows, and an output inside a wider buffer."""
    a, b = i8((M, K), 13), i8((N, K), 14)
    a_s, b_s = np.full(M, 0.01, np.float32), np.full(N, 0.02, np.float32)
    pad = K + (1 if how == "odd" else 16 - K % 16 + 16)
    off = {"odd": 3, "wide": 0, "offset16": 16}[how]
    c = strided(M, N, N + (5 if how == "odd" else 8 - N % 8 + 8), 1 if how == "odd" else 8, torch.bfloat16)
    whole = c.as_strided((M, c.stride(0)), (c.stride(0), 1))
    whole.fill_(7.0)
    ds.gemm_i8(dev_i8(a, pad, off), torch.from_numpy(a_s).cuda(), dev_i8(b, pad, off), torch.from_numpy(b_s).cuda(),
               out=c)
    assert np.array_equal(host_bits16(c), Q8.gemm(a, a_s, b, b_s))
    assert bool((whole[:, N:] == 7.0).all()), "elements between rows were written"


def test_gemm_extreme_sums():
    """The largest K the call takes, with sums near the ends of 32 bits."""
    K = 131071
    a = np.full((3, K), -128, np.int8)
    a[1], a[2, ::2] = 127, 127
    b = np.full((2, K), -128, np.int8)
    b[1] = 127
    one = np.ones(3, np.float32)
    c = ds.gemm_i8(dev_i8(a), torch.ones(3, device="cuda"), dev_i8(b), torch.ones(2, device="cuda"))
    assert np.array_equal(host_bits16(c), Q8.gemm(a, one, b, one[:2]))


def test_gemm_weight_past_4_gib():
    """Row offsets of the weight past 32 bits: the last rows of a 4.3 GB weight."""
    N, K, M = 270000, 16000, 2
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    tail = i8((40, K), 15)
    w[-40:] = torch.from_numpy(tail).cuda()
    a = i8((M, K), 16)
    c = ds.gemm_i8(dev_i8(a), torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"))
    ref = Q8.gemm(a, np.ones(M, np.float32), tail, np.ones(40, np.float32))
    assert np.array_equal(host_bits16(c[:, -40:]), ref)
    assert bool((c[:, :-40] == 0).all())


LINEARS = [(1, 64, 64), (1, 1536, 7168), (2, 300, 1000), (4, 100, 20000), (8, 513, 129), (16, 512, 1024), (17, 1536, 7168),
           (64, 7168, 2048), (333, 2500, 1000), (700, 1100, 640), (1, 5, 3), (5, 18432, 512), (6, 33, 0), (3, 16, 40000)]


@pytest.mark.parametrize("M,N,K", LINEARS)
def test_linear_bit_exact(M, N, K):
    x = bits((M, K), 20, outliers=0.01)
    b = i8((N, K), 21)
    b_s = I.rng(CID, 22).uniform(1e-4, 2e-4, N).astype(np.float32)
    c = ds.linear_i8(dev_bf16(x), dev_i8(b), torch.from_numpy(b_s).cuda())
    assert np.array_equal(host_bits16(c), Q8.linear(x, b, b_s))


@pytest.mark.parametrize("M,N,K", [(1, 128, 512), (3, 77, 2049), (8, 300, 1000), (40, 512, 714), (300, 600, 1024)])
def test_linear_forms_agree(M, N, K):
    """Both linear forms equal the quantiser followed by the product, byte for byte, from strided inputs."""
    g, u = (strided(M, K, 2 * K + 3, o, torch.bfloat16) for o in (1, 2))
    g.copy_(dev_bf16(bits((M, K), 23)))
    u.copy_(dev_bf16(bits((M, K), 24)))
    w, w_s = ds.row_quant_i8(torch.from_numpy(I.weights_f32((N, K), CID, 25)).cuda())
    assert torch.equal(ds.linear_i8(g, w, w_s), ds.gemm_i8(*ds.row_quant_i8(g), w, w_s))
    assert torch.equal(ds.silu_mul_linear_i8(g, u, w, w_s), ds.gemm_i8(*ds.silu_mul_row_quant_i8(g, u), w, w_s))


def test_linear_bad_rows_stay_their_own():
    M, N, K = 6, 200, 512
    x = dev_bf16(bits((M, K), 26))
    w, w_s = ds.row_quant_i8(torch.from_numpy(I.weights_f32((N, K), CID, 27)).cuda())
    good = ds.linear_i8(x, w, w_s)
    x[2, 100], x[4, 0] = float("nan"), float("-inf")
    c = ds.linear_i8(x, w, w_s)
    assert not bool(torch.isfinite(c[2]).any()) and not bool(torch.isfinite(c[4]).any())
    keep = [0, 1, 3, 5]
    assert torch.equal(c[keep], good[keep])


def test_linear_on_another_stream_and_graph():
    M, N, K = 3, 640, 1024
    x = dev_bf16(bits((M, K), 28))
    w, w_s = ds.row_quant_i8(torch.from_numpy(I.weights_f32((N, K), CID, 29)).cuda())
    big = torch.randn(400, K, device="cuda").to(torch.bfloat16)
    out = [torch.empty((n, N), dtype=torch.bfloat16, device="cuda") for n in (M, 400)]
    ws = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ds.linear_i8(x, w, w_s, out=out[0], workspace=ws[0])
    side.synchronize()
    assert torch.equal(out[0], ds.linear_i8(x, w, w_s))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.linear_i8(x, w, w_s, out=out[0], workspace=ws[0])
        ds.linear_i8(big, w, w_s, out=out[1], workspace=ws[1])
    for i in range(4):
        x.copy_(dev_bf16(bits((M, K), 30 + i)))
        big.mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], ds.linear_i8(x, w, w_s)) and torch.equal(out[1], ds.linear_i8(big, w, w_s))


def test_refusals():
    x = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((8, 32), dtype=torch.int8, device="cuda")
    s = torch.ones(8, device="cuda")
    with pytest.raises(ds.Dsfp8Error):
        ds.linear_i8(x.float(), w, s)
    with pytest.raises(ds.Dsfp8Error):
        ds.linear_i8(x, w, s[:7])
    with pytest.raises(ds.Dsfp8Error):
        ds.linear_i8(x[:, :31], w, s)
    with pytest.raises(ds.Dsfp8Error):
        ds.linear_i8(x.repeat(10, 1), w, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ds.Dsfp8Error):
        ds.linear_i8(x.t().contiguous().t(), w, s)
    with pytest.raises(ds.Dsfp8Error):
        ds.linear_i8(x, w.cpu(), s)
    with pytest.raises(ds.Dsfp8Error):
        ds.silu_mul_linear_i8(x, x[:3], w, s)
    with pytest.raises(ds.Dsfp8Error):
        ds.gemm_i8(w, s, w.view(torch.uint8), s)
    with pytest.raises(ds.Dsfp8Error):
        ds.gemm_i8(w, s, w, torch.ones(16, device="cuda")[::2])
    with pytest.raises(ds.Dsfp8Error):
        ds.row_quant_i8(x.half())
    with pytest.raises(ds.Dsfp8Error):
        ds.silu_mul_row_quant_i8(x, x[:, :16])


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (3, 8, 20), (16, 33, 132), (20, 96, 500), (33, 50, 2044), (70, 260, 604),
                                   (100, 7000, 1004), (130, 1300, 36), (600, 700, 1028), (700, 4100, 516),
                                   (2000, 1100, 508), (2100, 4200, 260)])
def test_gemm_four_byte_alignment(M, N, K):
    """Rows that start at multiples of 4 bytes only, values beyond each row's end that must not count."""
    a, b = i8((M, K), 20), i8((N, K), 21)
    a_s, b_s = np.full(M, 0.01, np.float32), np.full(N, 0.02, np.float32)
    da, db = dev_i8(a, K + 4 + (-K % 8), 4), dev_i8(b, K + 4, 12)
    for d in (da, db):
        rows, ld = d.shape[0], d.stride(0)
        d.as_strided((rows, ld - K), (ld, 1), d.storage_offset() + K).fill_(99)
    c = ds.gemm_i8(da, torch.from_numpy(a_s).cuda(), db, torch.from_numpy(b_s).cuda())
    assert np.array_equal(host_bits16(c), Q8.gemm(a, a_s, b, b_s))


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (2, 5000, 1004), (9, 40, 20), (40, 200, 1000)])
def test_linear_four_byte_alignment(M, N, K):
    x, w = bits((M, K), 22), i8((N, K), 23)
    w_s = np.full(N, 0.02, np.float32)
    c = ds.linear_i8(dev_bf16(x), dev_i8(w, K + 4, 4), torch.from_numpy(w_s).cuda())
    assert np.array_equal(host_bits16(c), Q8.linear(x, w, w_s))


def test_single_rows_and_columns_of_any_stride():
    """A row or a column cut out by a transpose is contiguous, whatever stride torch gives its other dimension."""
    K, N = 200, 40
    b = bits((1, K), 24)
    row = dev_bf16(b).reshape(K, 1).t()
    assert row.shape == (1, K) and row.stride() == (1, 1)
    w, w_s = i8((N, K), 25), np.full(N, 0.02, np.float32)
    dw, dw_s = dev_i8(w), torch.from_numpy(w_s).cuda()
    y, s = ds.row_quant_i8(row)
    yr, sr = Q8.row_quant(F.bf16_to_f32(b))
    assert np.array_equal(y.cpu().numpy(), yr) and np.array_equal(s.cpu().numpy(), sr)
    want = Q8.linear(b, w, w_s)
    assert np.array_equal(host_bits16(ds.linear_i8(row, dw, dw_s)), want)
    assert np.array_equal(host_bits16(ds.gemm_i8(y.reshape(K, 1).t(), s, dw, dw_s)), want)
    out = torch.empty((N, 1), dtype=torch.bfloat16, device="cuda").t()
    assert np.array_equal(host_bits16(ds.gemm_i8(y, s, dw, dw_s, out=out)), want)
    one = dw[:1].reshape(K, 1).t()
    assert np.array_equal(host_bits16(ds.gemm_i8(y, s, one, dw_s[:1])), want[:, :1])
    h, hs = ds.silu_mul_row_quant_i8(row, row)
    h0, hs0 = ds.silu_mul_row_quant_i8(row.contiguous().clone(), row.contiguous().clone())
    assert torch.equal(h, h0) and torch.equal(hs, hs0)
    column = dev_bf16(bits((K, 1), 26)).reshape(1, K).t()
    assert column.stride() == (1, K)
    yc, sc = ds.row_quant_i8(column)
    yr, sr = Q8.row_quant(F.bf16_to_f32(bits((K, 1), 26)))
    assert np.array_equal(yc.cpu().numpy(), yr) and np.array_equal(sc.cpu().numpy(), sr)


def test_silu_mul_accuracy_over_the_gate():
    """One value per row, which the row's scale shows: relative to it within (|g| + 8) 2^-23, and 2^-23 for the
    division by 127 and the scale's rounding."""
    g = F.f32_to_bf16(np.linspace(-86.0, 86.0, 345).astype(np.float32))
    M = g.size
    gs, us = np.zeros((M, 64), np.uint16), np.zeros((M, 64), np.uint16)
    gs[:, 17], us[:, 17] = g, F.f32_to_bf16(np.full(M, 2.0 ** 60, np.float32))
    _, s = ds.silu_mul_row_quant_i8(dev_bf16(gs), dev_bf16(us))
    h = np.abs(Q8.silu_mul(gs, us)).max(1)
    keep = h > 0
    assert keep.sum() >= M - 1
    got = s.cpu().numpy().astype(np.float64) * 127
    bound = (np.abs(F.bf16_to_f32(g).astype(np.float64)) + 8) * 2.0 ** -23 + 2.0 ** -23
    assert np.all((np.abs(got / np.maximum(h, 2.0 ** -100) - 1) <= bound)[keep])


def test_gemm_without_k_shows_bad_scales():
    """An empty sum is 0, and 0 times a scale that is not finite is NaN, as the formula has it."""
    a, b = (torch.empty((n, 0), dtype=torch.int8, device="cuda") for n in (2, 3))
    a_s, b_s = torch.ones(2, device="cuda"), torch.tensor([1.0, float("inf"), 2.0], device="cuda")
    c = ds.gemm_i8(a, a_s, b, b_s).float().cpu().numpy()
    assert not c[:, [0, 2]].any() and np.isnan(c[:, 1]).all()
