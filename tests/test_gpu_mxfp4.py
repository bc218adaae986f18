"""GPU checks of MXFP4 quantisation and products against the oracle.

Codes and scale bytes are compared bit for bit.  A product's bf16 output is within half a step of
bf16, 2^-8 of the value, and of the bound that oracle/mxfp4.py states for an fp32 sum.
"""

import ctypes

import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as ds
from block_scaled_fp8_act_amd import _lib
from block_scaled_fp8_act_amd import inputs as I
from oracle import int8 as Q8
from oracle import mxfp4 as MX
from oracle.formats import bf16_to_f32

from gpu_helpers import bf16_to_f64, dev_bf16, dev_u8, host_bits16, host_u8

pytestmark = pytest.mark.gpu

CID = 120


def normal(M, K, seed, std=1.0):
    return bf16_to_f32(I.activations((M, K), CID, seed, std=std))


def mx_dev(q, s):
    """Codes and scales on the device, the scales' padding filled with the NaN code."""
    M, kb = s.shape
    room = torch.full((M, (kb + 15) // 16 * 16), 255, dtype=torch.uint8, device="cuda")
    room[:, :kb] = dev_u8(s)
    return dev_u8(q), room[:, :kb]


def rows_of(M, K, seed):
    """MXFP4 rows with every code, zeros, and scales over many binades."""
    g = I.rng(CID, seed)
    kb = MX.blocks(K)
    codes = g.integers(0, 16, (M, 32 * kb)).astype(np.uint8)
    codes[:, K:] = 0
    codes[g.random((M, 32 * kb)) < 0.1] = 0
    return MX.pack(codes), g.integers(118, 131, (M, kb)).astype(np.uint8)


def check_product(got, a, a_s, b, b_s, what=""):
    ref, bound = MX.gemm(a, a_s, b, b_s)
    C = bf16_to_f64(host_bits16(got))
    err = np.abs(C - ref)
    lim = (np.abs(ref) + bound) * 2.0 ** -8 + bound
    worst = float((err / np.where(lim > 0, lim, 1)).max()) if err.size else 0.0
    assert np.all(err <= lim), f"{what}: {worst:.3f} of the bound"


# ---- quantisation -----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 100), (17, 512), (333, 1000), (64, 7168), (7, 2049)])
def test_quant_bits(M, K, dtype):
    g = I.rng(CID, M * 7 + K)
    x = torch.from_numpy((g.standard_normal((M, K)) * np.exp2(g.integers(-60, 60, (M, 1)))).astype(np.float32)).to(dtype)
    x[0, 0] = -0.0
    q, s = ds.mxfp4_quant(x.cuda())
    qr, sr = MX.quant(x.double().numpy())
    assert np.array_equal(host_u8(s), sr)
    assert np.array_equal(host_u8(q), qr)
    v = ds.mxfp4_dequant(q, s, K)
    assert np.array_equal(bf16_to_f64(host_bits16(v)), MX.values(qr, sr, K))


def test_every_bf16_value_against_every_top():
    """Blocks whose largest value runs through every exponent, the others through every bf16 below it."""
    bits = np.arange(0, 0x7f80, 31, dtype=np.uint16)
    tops = (np.arange(1, 255, dtype=np.uint32) << 7).astype(np.uint16)          # 2^-126 .. 2^127
    x = np.tile(bits, (len(tops), 1))
    x = np.where(x > tops[:, None], 0x8000 | (x & 0x7f), x)
    pad = -x.shape[1] % 31
    x = np.concatenate([x, np.zeros((len(tops), pad), np.uint16)], 1).reshape(len(tops), -1, 31)
    x = np.concatenate([np.broadcast_to(tops[:, None, None], x.shape[:2] + (1,)), x], 2).reshape(len(tops), -1)
    q, s = ds.mxfp4_quant(dev_bf16(x))
    qr, sr = MX.quant(bf16_to_f32(x))
    assert np.array_equal(host_u8(s), sr) and np.array_equal(host_u8(q), qr)


def test_every_bf16_value_of_every_scale():
    """For each scale (the largest value of each of bf16's binades, and of its subnormals, at the head of every block) all
    bf16 values of either sign up to that largest one."""
    for first in range(0, 255, 15):
        rows = []
        for f in range(first, first + 15):
            v = np.arange((f + 1) << 7, dtype=np.uint16)
            v = np.concatenate([v, v | 0x8000])
            v = np.concatenate([v, np.zeros(-len(v) % 31, np.uint16)]).reshape(-1, 31)
            rows.append(np.concatenate([np.full((len(v), 1), (f << 7) | 0x7f, np.uint16), v], 1))
        x = np.concatenate(rows)
        q, s = ds.mxfp4_quant(dev_bf16(x))
        qr, sr = MX.quant(bf16_to_f32(x))
        assert np.array_equal(host_u8(s), sr) and np.array_equal(host_u8(q), qr), first


def test_halfway_cases_and_subnormals():
    steps = np.concatenate([MX.HALFWAY, np.nextafter(MX.HALFWAY.astype(np.float32), np.float32(0)),
                            np.nextafter(MX.HALFWAY.astype(np.float32), np.float32(9)), [0, 6, 7, 7.9, 0.1]])
    row = np.concatenate([[4.0], steps, -steps])
    row = np.concatenate([row, np.zeros(-len(row) % 32)])
    # every scale that leaves the values exact in fp32 (their last bits are 2^-26 of the scale), and the smallest
    x = np.stack([row * 2.0 ** e for e in list(range(-100, 124, 7)) + [-126, -127, -130, -147]]).astype(np.float32)
    x = np.concatenate([x, np.zeros((1, x.shape[1]), np.float32), np.full((1, x.shape[1]), 2.0 ** -149, np.float32)])
    q, s = ds.mxfp4_quant(torch.from_numpy(x).cuda())
    qr, sr = MX.quant(x)
    assert np.array_equal(host_u8(s), sr) and np.array_equal(host_u8(q), qr)
    # every value of every scale in bf16
    codes = np.tile(MX.pack(np.tile(np.arange(16, dtype=np.uint8), 2)), (256, 1))
    sc = np.arange(256, dtype=np.uint8)[:, None]
    got = bf16_to_f64(host_bits16(ds.mxfp4_dequant(*mx_dev(codes, sc))))
    want = MX.values(codes, sc)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
    np.testing.assert_array_equal(got, want)


def test_bad_values_stay_in_their_block():
    x = normal(6, 200, 5)
    x[1, 40], x[2, 199], x[3, 0] = np.nan, np.inf, -np.inf
    q, s = ds.mxfp4_quant(torch.from_numpy(x).cuda())
    qr, sr = MX.quant(x)
    assert np.array_equal(host_u8(s), sr)
    v = bf16_to_f64(host_bits16(ds.mxfp4_dequant(q, s, 200)))
    np.testing.assert_array_equal(v, MX.values(qr, sr, 200))
    b, bs = rows_of(40, 200, 6)
    c = bf16_to_f64(host_bits16(ds.gemm_mxfp4(q, s, *mx_dev(b, bs))))
    assert np.isnan(c[1:4]).all() and np.isfinite(c[[0, 4, 5]]).all()


@pytest.mark.parametrize("M,K", [(1, 32), (3, 50), (40, 2048), (5, 4099)])
def test_gated_quant(M, K):
    """x is within (|g| + 8) 2^-23 of SiLU(g) * u, so a code is that of a value in that range."""
    gb, ub = I.activations((M, K), CID, 30 + M, std=3.0), I.activations((M, K), CID, 31 + M)
    q, s = ds.silu_mul_mxfp4_quant(dev_bf16(gb), dev_bf16(ub))
    x = Q8.silu_mul(gb, ub)
    d = (np.abs(bf16_to_f32(gb).astype(np.float64)) + 8) * 2.0 ** -23
    kb = MX.blocks(K)

    def block_max(v):
        return np.pad(np.abs(v), ((0, 0), (0, 32 * kb - K))).reshape(M, kb, 32).max(axis=2)
    s = host_u8(s)
    assert np.all((s == MX.scale_byte(block_max(x * (1 - d)))) | (s == MX.scale_byte(block_max(x * (1 + d)))))
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)[:, :K]
    codes = MX.unpack(host_u8(q))
    assert not codes[:, K:].any()
    codes = codes[:, :K]
    assert np.all((codes == MX.encode(x * (1 - d) / unit)) | (codes == MX.encode(x * (1 + d) / unit)))


def test_quant_strides_and_untouched_padding():
    x = normal(9, 300, 7)
    big = torch.zeros((9, 331), device="cuda")
    big[:, 3:303] = torch.from_numpy(x).cuda()
    q = torch.full((9, 160 + 32), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((9, 32), 78, dtype=torch.uint8, device="cuda")
    ds.mxfp4_quant(big[:, 3:303], out=(q[:, :160], s[:, :10]))
    qr, sr = MX.quant(x)
    assert np.array_equal(host_u8(q[:, :160]), qr) and np.array_equal(host_u8(s[:, :10]), sr)
    assert (q[:, 160:] == 77).all() and (s[:, 10:] == 78).all()
    b16 = big.to(torch.bfloat16)
    q2, s2 = ds.mxfp4_quant(b16[:, 3:303])
    assert np.array_equal(host_u8(q2), MX.quant(b16[:, 3:303].cpu().double().numpy())[0])
    out = torch.full((9, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    ds.mxfp4_dequant(q2, s2, 300, out=out[:, 1:301])
    assert torch.equal(out[:, 1:301], ds.mxfp4_dequant(q2, s2, 300)) and (out[:, 301:] == 5).all() and (out[:, 0] == 5).all()


@pytest.mark.parametrize("gated", [False, True])
def test_quant_into_one_given_output(gated):
    x = dev_bf16(I.activations((9, 300), CID, 8))
    call = (lambda **kw: ds.silu_mul_mxfp4_quant(x, x, **kw)) if gated else (lambda **kw: ds.mxfp4_quant(x, **kw))
    ref = call()
    q, s = (t.fill_(9) for t in ds.mxfp4_empty(9, 300, "cuda"))
    got = call(out=(None, s))
    assert got[1].data_ptr() == s.data_ptr() and torch.equal(s, ref[1]) and torch.equal(got[0], ref[0])
    got = call(out=(q, None))
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, ref[0]) and torch.equal(got[1], ref[1])


def test_quant_of_more_rows_than_one_launch_takes():
    """2^28 + 5 rows of one block: two launches; the rows on both sides of the cut, and the last."""
    M = 2 ** 28 + 5
    x = torch.zeros((M, 1), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 7, 2 ** 28 - 1, 2 ** 28, M - 1], device="cuda")
    x[at, 0] = torch.tensor([1.0, -3.0, 0.5, 6.0, -40.0], dtype=torch.bfloat16, device="cuda")
    q, s = ds.mxfp4_quant(x)
    qr, sr = MX.quant(x[at].double().cpu().numpy())
    assert np.array_equal(host_u8(q[at]), qr) and np.array_equal(host_u8(s[at]), sr)
    assert int((q.view(M, 16)[:, 0] != 0).sum()) == 5
    del q, s
    torch.cuda.empty_cache()


# ---- products ---------------------------------------------------------------------------------

# one row or column, sizes around a block, around 256 columns of K (a K-block), 512 (two: one load of
# scales), around the tiles' 16, 64, 128 and 256 rows and columns, few and many tiles
SIZES = [(1, 1, 1), (1, 1, 32), (2, 3, 33), (16, 16, 256), (17, 15, 255), (5, 64, 257), (64, 64, 512), (65, 63, 513),
         (33, 130, 544), (1, 1536, 7168), (4, 300, 4096), (8, 100, 2880), (16, 257, 1024), (31, 72, 800), (32, 512, 2048),
         (100, 1000, 96), (128, 128, 1504), (129, 250, 64), (200, 1001, 1300), (333, 2500, 1000), (256, 256, 3584),
         (257, 511, 320), (3, 4100, 544), (700, 640, 1056)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm(M, N, K):
    a, a_s = rows_of(M, K, 1000 + M)
    b, b_s = rows_of(N, K, 2000 + N)
    A, B = mx_dev(a, a_s), mx_dev(b, b_s)
    c = ds.gemm_mxfp4(*A, *B)
    check_product(c, a, a_s, b, b_s, f"{M}x{N}x{K}")
    assert torch.equal(c, ds.gemm_mxfp4(*A, *B)), "the same call gives the same bytes"


@pytest.mark.parametrize("M,N,K", [(4096, 4100, 288), (2050, 8200, 768), (1000, 20000, 544)])
def test_gemm_many_tiles(M, N, K):
    """More 256x256 tiles than CUs, with ragged edges, on a sample of rows."""
    a, a_s = rows_of(M, K, 3000)
    b, b_s = rows_of(N, K, 3001)
    c = ds.gemm_mxfp4(*mx_dev(a, a_s), *mx_dev(b, b_s))
    pick = np.unique(np.concatenate([np.arange(0, M, 37), [M - 1, 255, 256]]))
    check_product(c[torch.from_numpy(pick).cuda()], a[pick], a_s[pick], b, b_s)


def tile(E, M, N, K):
    v = (ctypes.c_int32 * 2)()
    assert _lib.load().dsfp8_mxfp4_variant(E, M, N, K, ctypes.addressof(v)) == 0
    return tuple(v)


# tile, M, N, K: ragged edges, more tiles than workgroups for the larger ones, K of one K-block of 256 columns, of odd
# and even numbers of them, and ends inside one
VARIANTS = [((16, 16), 9, 300, 1000), ((16, 32), 9, 9000, 1000), ((16, 32), 40, 3000, 1000), ((32, 32), 64, 7200, 700),
            ((32, 32), 20, 9001, 1000), ((64, 64), 150, 9000, 700), ((64, 64), 300, 2100, 288), ((64, 64), 500, 3001, 1056),
            ((64, 128), 800, 2700, 1120), ((128, 128), 2048, 7168, 288), ((128, 128), 900, 5003, 1312),
            ((256, 256), 4000, 16300, 200), ((256, 256), 4000, 16300, 288), ((256, 256), 4090, 16201, 544),
            ((256, 256), 3000, 12000, 800), ((256, 256), 700, 20000, 1300)]


@pytest.mark.parametrize("want,M,N,K", VARIANTS)
def test_every_variant(want, M, N, K):
    assert tile(0, M, N, K) == want
    a, a_s = rows_of(M, K, 4000)
    b, b_s = rows_of(N, K, 4001)
    c = ds.gemm_mxfp4(*mx_dev(a, a_s), *mx_dev(b, b_s))
    pick = np.unique(np.concatenate([np.arange(0, M, max(1, M // 60)), [M - 1, M // 2]]))
    check_product(c[torch.from_numpy(pick).cuda()], a[pick], a_s[pick], b, b_s, f"{M}x{N}x{K}")


GROUPED = [((16, 32), [20, 0, 3, 60, 7], 1000, 1056), ((32, 32), [9, 14, 0, 33, 40, 1, 2, 29], 2100, 2336),
           ((64, 128), [0, 100, 64, 3, 90, 1, 0, 42], 8200, 544), ((128, 128), [130, 0, 1800, 70], 2100, 288),
           ((256, 256), [4000, 300, 4700], 8100, 288), ((256, 256), [257, 8743], 4101, 544),
           ((256, 256), [4000, 0, 256, 744], 8200, 1056)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("want,counts,N,K", GROUPED)
def test_every_grouped_variant(want, counts, N, K, gather):
    assert tile(len(counts), sum(counts), N, K) == want
    a, a_s, w, off, rows = grouped(counts, N, K, 600, 500 if gather else None)
    c = ds.grouped_gemm_mxfp4(*grouped_dev(a, a_s, w), torch.from_numpy(off).cuda(),
                              rows=None if rows is None else torch.from_numpy(rows).cuda())
    for e, (b, b_s) in enumerate(w):
        if counts[e]:
            r = np.unique(np.concatenate([np.arange(off[e], off[e + 1], max(1, counts[e] // 25)), [off[e + 1] - 1]]))
            src = r if rows is None else rows[r]
            check_product(c[torch.from_numpy(r).cuda()], a[src], a_s[src], b, b_s, f"expert {e}")


def test_gemm_small_whole_numbers_are_exact():
    """Sums of small whole numbers are exact in fp32 and, below 256, in bf16: every element, bit for bit."""
    g = I.rng(CID, 40)
    for M, N, K in [(40, 48, 512), (300, 520, 288), (16, 16, 1024)]:
        a, b = (MX.pack(np.where(g.random((r, K)) < 0.03, g.integers(0, 16, (r, K)) & 0xa, 0).astype(np.uint8)) for r in (M, N))
        s = [np.full((r, K // 32), 127, np.uint8) for r in (M, N)]
        ref = MX.gemm(a, s[0], b, s[1])[0]
        assert np.abs(ref).max() <= 256
        c = ds.gemm_mxfp4(*mx_dev(a, s[0]), *mx_dev(b, s[1]))
        assert np.array_equal(bf16_to_f64(host_bits16(c)), ref)


@pytest.mark.parametrize("M,N,K", [(20, 40, 320), (300, 300, 320), (4, 40, 320)])
def test_gemm_strides_and_offsets(M, N, K):
    """Operands inside larger buffers, C at an odd address with a stride, nothing else written."""
    a, a_s = rows_of(M, K, 50)
    b, b_s = rows_of(N, K, 51)

    def inside(q, s):
        Q = torch.full((len(q), q.shape[1] + 48), 255, dtype=torch.uint8, device="cuda")
        S = torch.full((len(s), 64), 255, dtype=torch.uint8, device="cuda")
        Q[:, 16:16 + q.shape[1]] = dev_u8(q)
        S[:, 16:16 + s.shape[1]] = dev_u8(s)
        return Q[:, 16:16 + q.shape[1]], S[:, 16:16 + s.shape[1]]
    C = torch.full((M + 2, N + 7), 3.0, dtype=torch.bfloat16, device="cuda")
    ds.gemm_mxfp4(*inside(a, a_s), *inside(b, b_s), out=C[1:M + 1, 3:N + 3])
    check_product(C[1:M + 1, 3:N + 3], a, a_s, b, b_s)
    C[1:M + 1, 3:N + 3] = 3
    assert (C == 3).all()


def test_gemm_nan_scales():
    """The scale byte 255 on either side makes NaN of its rows or columns and of nothing else."""
    for M, N, K in [(40, 50, 600), (400, 300, 600), (2, 50, 600)]:
        a, a_s = rows_of(M, K, 60)
        b, b_s = rows_of(N, K, 61)
        a_s[1, 18], b_s[7, 0] = 255, 255
        c = bf16_to_f64(host_bits16(ds.gemm_mxfp4(*mx_dev(a, a_s), *mx_dev(b, b_s))))
        nan = np.zeros((M, N), bool)
        nan[1], nan[:, 7] = True, True
        assert np.array_equal(np.isnan(c), nan)


@pytest.mark.parametrize("M,N,K", [(3, 40, 320), (40, 50, 600), (300, 300, 320), (900, 5003, 320), (3000, 12000, 288)])
def test_gemm_scales_at_the_ends_of_their_range(M, N, K):
    """A block's two scales meet as one power of two, whatever they are alone.  Below 2^-126 bf16's values are 2^-133
    apart, so the output's rounding is off by up to 2^-134 there."""
    a, _ = rows_of(M, K, 65)
    b, _ = rows_of(N, K, 66)
    for ea, eb in [(0, 254), (254, 0), (1, 253), (0, 150), (254, 60), (20, 100), (60, 60), (0, 0)]:
        a_s, b_s = np.full((M, MX.blocks(K)), ea, np.uint8), np.full((N, MX.blocks(K)), eb, np.uint8)
        c = bf16_to_f64(host_bits16(ds.gemm_mxfp4(*mx_dev(a, a_s), *mx_dev(b, b_s))[-50:, -50:]))
        ref, bound = MX.gemm(a[-50:], a_s[-50:], b[-50:], b_s[-50:])
        assert np.all(np.abs(c - ref) <= (np.abs(ref) + bound) * 2.0 ** -8 + bound + 2.0 ** -134), (ea, eb)


def test_torch_types_of_codes_and_scales():
    """torch's own types for two e2m1 codes a byte and for powers of two are taken as bytes."""
    f4, e8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
    (a, a_s), (b, b_s) = (mx_dev(*rows_of(r, 320, 67)) for r in (70, 48))
    ref = ds.gemm_mxfp4(a, a_s, b, b_s)
    assert torch.equal(ref, ds.gemm_mxfp4(a.view(f4), a_s.view(e8), b.view(f4), b_s.view(e8)))
    assert torch.equal(ref, ds.gemm_mxfp4(a, a_s, b.view(f4), b_s))
    assert torch.equal(ds.mxfp4_dequant(a, a_s, 300), ds.mxfp4_dequant(a.view(f4), a_s.view(e8), 300))
    x = torch.randn((2, 320), device="cuda").bfloat16()
    assert torch.equal(ds.linear_mxfp4(x, b, b_s), ds.linear_mxfp4(x, b.view(f4), b_s.view(e8)))


def test_empty_products():
    for M, N in [(0, 5), (5, 0)]:
        assert ds.gemm_mxfp4(*ds.mxfp4_empty(M, 64, "cuda"), *ds.mxfp4_empty(N, 64, "cuda")).shape == (M, N)
    c = torch.ones((70, 9), dtype=torch.bfloat16, device="cuda")
    ds.gemm_mxfp4(*ds.mxfp4_empty(70, 0, "cuda"), *ds.mxfp4_empty(9, 0, "cuda"), out=c)
    assert not c.any()
    q, s = ds.mxfp4_quant(torch.empty((4, 0), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (4, 0) and s.shape == (4, 0)
    for M in (1, 40):
        c = ds.linear_mxfp4(torch.empty((M, 0), dtype=torch.bfloat16, device="cuda"), *ds.mxfp4_empty(9, 0, "cuda"))
        assert c.shape == (M, 9) and not c.any()


# ---- linear -----------------------------------------------------------------------------------


@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (1, 1536, 7168), (2, 100, 1000), (3, 130, 2049), (4, 64, 8192), (7, 48, 4095),
                                   (8, 257, 1), (9, 33, 600), (16, 200, 2048), (16, 31, 5000), (17, 64, 512),
                                   (40, 500, 1030), (300, 200, 700), (1, 40, 18432)])
def test_linear_equals_its_steps(M, N, K):
    xb = I.activations((M, K), CID, 70 + M, outlier_frac=0.02)
    b, b_s = rows_of(N, K, 71)
    B = mx_dev(b, b_s)
    x = dev_bf16(xb)
    a, a_s = MX.quant(bf16_to_f32(xb))
    c = ds.linear_mxfp4(x, *B)
    check_product(c, a, a_s, b, b_s)
    need = ds.linear_mxfp4_workspace_bytes(M, N, K)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")[:need]
    assert torch.equal(c, ds.linear_mxfp4(x, *B, workspace=ws))
    wide = torch.zeros((M, K + 5), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:K + 3] = x
    assert torch.equal(c, ds.linear_mxfp4(wide[:, 3:K + 3], *B))


@pytest.mark.parametrize("M,N,K", [(1, 4100, 2048), (1, 4097, 7168), (2, 9001, 1000), (3, 18433, 1031), (5, 4500, 4800),
                                   (16, 5000, 1500)])
def test_linear_in_one_launch_with_many_columns(M, N, K):
    """Few rows and more than 16 columns for every CU: 32 columns a workgroup, the last tile ragged, K ending inside a
    K-block of 256 or with one."""
    assert ds.linear_mxfp4_workspace_bytes(M, N, K) == 0
    assert N > 16 * torch.cuda.get_device_properties(0).multi_processor_count
    xb = I.activations((M, K), CID, 170 + M, outlier_frac=0.02)
    b, b_s = rows_of(N, K, 171)
    B = mx_dev(b, b_s)
    a, a_s = MX.quant(bf16_to_f32(xb))
    C = torch.full((M + 2, N + 9), 5.0, dtype=torch.bfloat16, device="cuda")
    c = ds.linear_mxfp4(dev_bf16(xb), *B, out=C[1:M + 1, 5:N + 5])
    check_product(c, a, a_s, b, b_s)
    assert torch.equal(c, ds.linear_mxfp4(dev_bf16(xb), *B))
    c.fill_(5)
    assert (C == 5).all()


def test_linear_nan_row():
    for M in (3, 40):
        x = I.activations((M, 700), CID, 80)
        x[1, 699] = 0x7fc0
        b, b_s = rows_of(40, 700, 81)
        c = bf16_to_f64(host_bits16(ds.linear_mxfp4(dev_bf16(x), *mx_dev(b, b_s))))
        assert np.isnan(c[1]).all() and np.isfinite(np.delete(c, 1, 0)).all()


# ---- grouped ----------------------------------------------------------------------------------


def grouped(counts, N, K, seed, a_rows=None):
    """Operands of a grouped product; with a_rows, rows read through an index."""
    E, M = len(counts), int(sum(counts))
    g = I.rng(CID, seed)
    a, a_s = rows_of(M if a_rows is None else a_rows, K, seed + 1)
    w = [rows_of(N, K, seed + 2 + e) for e in range(E)]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = None if a_rows is None else g.integers(0, a_rows, M).astype(np.int32)
    return a, a_s, w, off, rows


def grouped_dev(a, a_s, w):
    W = [mx_dev(*p) for p in w]
    kb = a_s.shape[1]
    q = torch.stack([v[0] for v in W])
    room = torch.full((len(W), W[0][1].shape[0], (kb + 15) // 16 * 16), 255, dtype=torch.uint8, device="cuda")
    for e, v in enumerate(W):
        room[e, :, :kb] = v[1]
    return (*mx_dev(a, a_s), q, room[..., :kb])


COUNTS = [[1], [5, 0, 17], [0, 0, 3], [16, 1, 1, 0, 33, 2], [64, 65, 1, 0, 128], [130, 0, 300, 7], [0] * 70 + [3] + [0] * 9 + [1],
          [1] * 100, [700, 20]]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(72, 288), (300, 1056)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped(counts, N, K, gather):
    a, a_s, w, off, rows = grouped(counts, N, K, 300, 23 if gather else None)
    dev = grouped_dev(a, a_s, w)
    offd = torch.from_numpy(off).cuda()
    rd = None if rows is None else torch.from_numpy(rows).cuda()
    c = ds.grouped_gemm_mxfp4(*dev, offd, rows=rd)
    assert torch.equal(c, ds.grouped_gemm_mxfp4(*dev, offd, rows=rd))
    for e, (b, b_s) in enumerate(w):
        r = np.arange(off[e], off[e + 1])
        if len(r):
            src = r if rows is None else rows[r]
            check_product(c[off[e]:off[e + 1]], a[src], a_s[src], b, b_s, f"expert {e}")


def test_grouped_rows_of_no_expert_are_left():
    """Rows past the last expert (another rank's) and indices outside the token rows (clamped)."""
    a, a_s, w, off, rows = grouped([3, 40, 0, 9], 80, 320, 400, 10)
    rows = np.concatenate([rows, np.full(30, 2 ** 31 - 1)]).astype(np.int32)
    rows[0], rows[1] = -5, 99
    c = torch.full((len(rows), 80), 7.0, dtype=torch.bfloat16, device="cuda")
    ds.grouped_gemm_mxfp4(*grouped_dev(a, a_s, w), torch.from_numpy(off).cuda(), rows=torch.from_numpy(rows).cuda(), out=c)
    assert (c[52:] == 7).all()
    src = np.clip(rows[:3], 0, 9)
    check_product(c[:3], a[src], a_s[src], *w[0])


def test_grouped_malformed_offsets_stay_inside():
    """Offsets out of order or out of range: nothing outside C is written, and the ranges that are well formed hold."""
    a, a_s, w, _, _ = grouped([4, 4, 4, 4], 40, 96, 500)
    dev = grouped_dev(a, a_s, w)
    C = torch.full((16 + 8, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, 4, -3, 8, 2 ** 31 - 1], [-2 ** 31, 100, 3, 2, 1], [16, 16, 16, 16, 16], [0, 16, 0, 16, 0]):
        ds.grouped_gemm_mxfp4(*dev, torch.tensor(off, dtype=torch.int32, device="cuda"), out=C[4:20])
        torch.cuda.synchronize()
        assert (C[:4] == 7).all() and (C[20:] == 7).all()


# ---- streams, graphs, refusals -----------------------------------------------------------------


def test_other_stream_and_graph():
    """A captured pass of quantiser, products and grouped product, replayed with new inputs between replays."""
    M, N, K = 48, 320, 544
    b, b_s = rows_of(N, K, 90)
    B = mx_dev(b, b_s)
    room = torch.zeros((1, N, 32), dtype=torch.uint8, device="cuda")
    room[0, :, :17] = B[1]
    W = (B[0][None], room[..., :17])
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    x = dev_bf16(I.activations((M, K), CID, 91))
    ws = torch.empty(ds.linear_mxfp4_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    qs = ds.mxfp4_empty(M, K, "cuda")
    outs = [torch.empty((m, N), dtype=torch.bfloat16, device="cuda") for m in (M, M, M, 2)]

    def step():
        ds.mxfp4_quant(x, out=qs)
        ds.gemm_mxfp4(*qs, *B, out=outs[0])
        ds.linear_mxfp4(x, *B, out=outs[1], workspace=ws)
        ds.grouped_gemm_mxfp4(*qs, *W, off, out=outs[2])
        ds.linear_mxfp4(x[:2], *B, out=outs[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(4):
        xb = I.activations((M, K), CID, 92 + seed)
        x.copy_(dev_bf16(xb))
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, outs))
        a, a_s = MX.quant(bf16_to_f32(xb))
        for o in outs[:3]:
            check_product(o, a, a_s, b, b_s)
        check_product(outs[3], a[:2], a_s[:2], b, b_s)


def test_weight_past_4_gib():
    """Rows of codes more than 2^32 bytes from the base."""
    N, K = 600000, 16384
    q, s = ds.mxfp4_empty(N, K, "cuda")
    q.zero_()
    s.fill_(127)
    a, a_s = rows_of(3, K, 95)
    b, b_s = rows_of(50, K, 96)
    q[-50:], s[-50:] = dev_u8(b), dev_u8(b_s)
    c = ds.gemm_mxfp4(*mx_dev(a, a_s), q, s)
    assert not c[:, :-50].any()
    check_product(c[:, -50:], a, a_s, b, b_s)
    x = torch.zeros((3, K), dtype=torch.bfloat16, device="cuda")
    assert not ds.linear_mxfp4(x, q, s).any()
    v = ds.mxfp4_dequant(q[-3:], s[-3:])
    assert np.array_equal(bf16_to_f64(host_bits16(v)), MX.values(b[-3:], b_s[-3:]))


def test_refusals():
    q, s = ds.mxfp4_empty(4, 64, "cuda")
    E = ds.Dsfp8Error
    tight = torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    for bad in (lambda: ds.gemm_mxfp4(q, tight, q, s), lambda: ds.gemm_mxfp4(q, s, q, tight),
                lambda: ds.mxfp4_dequant(q, tight), lambda: ds.mxfp4_dequant(q, s, 32), lambda: ds.mxfp4_dequant(q, s, 65),
                lambda: ds.gemm_mxfp4(q, s[:3], q, s), lambda: ds.gemm_mxfp4(q[:, :16], s, q, s),
                lambda: ds.gemm_mxfp4(q, s, *ds.mxfp4_empty(4, 96, "cuda")), lambda: ds.gemm_mxfp4(q.cpu(), s, q, s),
                lambda: ds.gemm_mxfp4(q.int(), s, q, s), lambda: ds.mxfp4_quant(torch.zeros((2, 2), device="cuda").half()),
                lambda: ds.mxfp4_quant(torch.zeros((2, 2))), lambda: ds.mxfp4_quant(torch.zeros((2, 64), device="cuda"), out=(q, s)),
                lambda: ds.mxfp4_quant(torch.zeros((4, 64), device="cuda"), out=(q, tight)),
                lambda: ds.linear_mxfp4(torch.zeros((2, 65), dtype=torch.bfloat16, device="cuda"), q, s),
                lambda: ds.linear_mxfp4(torch.zeros((2, 64), device="cuda"), q, s),
                lambda: ds.linear_mxfp4(torch.zeros((200, 64), dtype=torch.bfloat16, device="cuda"), q, s,
                                        workspace=torch.empty(3, dtype=torch.uint8, device="cuda")),
                lambda: ds.grouped_gemm_mxfp4(q, s, q[None], s[None], torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: ds.grouped_gemm_mxfp4(q, s, q[None], s[None], torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: ds.silu_mul_mxfp4_quant(*(torch.zeros((2, n), dtype=torch.bfloat16, device="cuda") for n in (3, 4)))):
        with pytest.raises(E):
            bad()
    # a view whose last row has no room for its 16 bytes of scales
    flat = torch.zeros(3 * 16 + 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(E):
        ds.mxfp4_dequant(q, flat.as_strided((4, 2), (16, 1)))
