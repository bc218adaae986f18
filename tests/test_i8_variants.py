"""Every kernel of the int8 product, reached by a case that is shown to select it.

The case lists name the kernel that serves each case; that the library would
choose it is checked on the host (256 CUs), and the GPU tests check it again
before they compare the product bit for bit.  The reference is a torch product
in float64 (the sums are whole numbers below 2^53, so exact in any order), the
definition's two float32 multiplications and the rounding to bf16.
"""

import ctypes
import os

import pytest
import torch

from block_scaled_fp8_act_amd import _lib

NONE, TILES, SPLIT, FUSED, SHORT = range(5)
WIDE, DWORD, SHIFT, REGS = 16, 4, 1, 0      # bytes per lane and load; aligned dwords of the weight; registers

# Tile and a product that takes it, ragged in both directions.
AT = {(64, 64): (65, 4101), (128, 128): (260, 7001), (128, 256): (520, 7001), (256, 256): (2000, 4101)}
WALK = (5117, 5115)     # 20 x 20 tiles of 256x256: workgroups of 256 CUs walk to a second tile, some to none


def _gemm_tiles():
    for tile, (M, N) in AT.items():
        for feed, sizes in ((WIDE, (256, 640, 1152, 144, 400, 656)), (DWORD, (260, 388, 1156)),
                            (REGS, (513, 1151) if tile == (64, 64) else (257, 385, 1151))):
            for K in sizes:
                m = 100 if tile == (64, 64) and (feed == DWORD or K in (400, 640, 656)) else M
                yield (m, N, K, feed) + tile
    # fewer than one K-block, and one
    yield from [(100, 4101, 60, DWORD, 64, 64), (33, 4101, 48, WIDE, 64, 64), (200, 4101, 128, WIDE, 128, 128),
                (200, 4101, 60, DWORD, 128, 128), (17, 4101, 61, REGS, 128, 128), (520, 7001, 48, WIDE, 128, 256),
                (520, 7001, 127, REGS, 128, 256), (520, 7001, 132, DWORD, 128, 256), (2000, 4101, 128, WIDE, 256, 256),
                (2000, 4101, 129, REGS, 256, 256)]
    M, N = WALK
    for feed, sizes in ((WIDE, (128, 256, 384, 1024, 112, 144, 400)), (DWORD, (124, 132, 388, 1036)),
                        (REGS, (127, 257, 385, 1025))):
        for K in sizes:
            yield M, N, K, feed, 256, 256


GEMM_TILES = list(_gemm_tiles())

GEMM_SPLIT = [(17, 50, 128, WIDE, 16, 8), (17, 50, 1168, WIDE, 16, 8), (17, 1100, 1024, WIDE, 16, 16),
              (17, 4101, 1024, WIDE, 32, 32), (33, 4101, 656, WIDE, 64, 32), (100, 4101, 1024, WIDE, 64, 64),
              (17, 50, 1028, DWORD, 16, 8), (17, 51, 132, DWORD, 16, 16), (17, 4101, 132, DWORD, 32, 32),
              (333, 2500, 1000, DWORD, 64, 64), (17, 50, 1153, REGS, 16, 8), (17, 2101, 1153, REGS, 16, 16),
              (17, 4101, 131, REGS, 32, 32), (4200, 50, 1001, REGS, 64, 32)]


def _linear_tiles():
    """Weights at any address: the row's end at every place in a dword and at both sides of a K-block's end (K modulo
    128 of 0, 1, 2, 3, 125, 126, 127), the first row's address and the row stride at every residue modulo 4."""
    for tile, (M, N) in AT.items():
        for i, K in enumerate((129, 253, 254, 255, 256, 257, 258, 259, 513, 641, 1149, 1151, 1277)):
            if tile == (64, 64) and K < 513:
                m = 33
            elif tile == (64, 64) and K == 513:
                m = 65
            else:
                m = {(128, 128): 200}.get(tile, M)
            n = N if tile != (128, 128) else 4101
            offset, ld = i % 4, K + 1 + i // 4      # 13 cases: all pairs of residues but three
            if (offset | ld) % 4 == 0:
                offset = 1
            yield (m, n, K, offset, ld) + tile
    for K, offset, ld in ((61, 1, 61), (61, 3, 64), (125, 2, 127), (127, 0, 127), (128, 3, 128)):
        yield 17 if K < 128 else 200, 4101, K, offset, ld, 128, 128
        yield 520, 7001, K, offset, ld, 128, 256
        yield 2000, 4101, K, offset, ld, 256, 256
    M, N = WALK
    for K, offset, ld in ((127, 1, 127), (127, 2, 130), (128, 1, 132), (129, 0, 131), (255, 3, 257), (255, 0, 255),
                          (385, 2, 386), (383, 3, 383), (1021, 1, 1023)):
        yield M, N, K, offset, ld, 256, 256


LINEAR_TILES = list(_linear_tiles())

# call (1 plain, 2 gated), M, N, K, feed, columns: one launch with the quantisation.  15 x 1088 has more than the 32
# units of 64 chunks that the waves hold at once.
FUSED_CASES = [(1, 1, 1536, 7168, WIDE, 8), (1, 1, 700, 16384, WIDE, 8), (1, 15, 100, 1088, WIDE, 8),
               (1, 16, 301, 529, REGS, 8), (1, 3, 77, 2052, DWORD, 8), (1, 8, 5001, 1024, WIDE, 16),
               (1, 7, 5001, 1028, DWORD, 16), (1, 8, 5001, 1021, REGS, 16), (1, 16, 4100, 16, WIDE, 16),
               (2, 4, 1000, 2048, WIDE, 8), (2, 15, 100, 528, WIDE, 8), (2, 15, 301, 545, REGS, 8),
               (2, 3, 77, 2052, DWORD, 8), (2, 4, 5001, 1024, WIDE, 16), (2, 3, 5001, 1028, DWORD, 16),
               (2, 4, 5001, 1021, REGS, 16), (2, 16, 4100, 17, REGS, 16)]


def variant(call, M, N, K, lda=0, a_offset=0, ldb=0, b_offset=0):
    """(kind, rows, columns, feed) of a call whose operands start so many bytes past a 16-byte boundary."""
    v = (ctypes.c_int32 * 4)()
    st = _lib.load().dsfp8_i8_variant(call, 4096 + a_offset, lda or K, 4096 + b_offset, ldb or K, M, N, K, v)
    assert st == 0
    return tuple(v)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from block_scaled_fp8_act_amd import build
        build.build()
    return _lib.load()


# ---- on the host ---------------------------------------------------------------------------


def test_selection():
    for M, N, K, feed, rows, cols in GEMM_TILES:
        assert variant(0, M, N, K) == (TILES, rows, cols, feed), (M, N, K)
    for M, N, K, feed, rows, cols in GEMM_SPLIT:
        assert variant(0, M, N, K) == (SPLIT, rows, cols, feed), (M, N, K)
    for M, N, K, offset, ld, rows, cols in LINEAR_TILES:
        for call in (1, 2):
            assert variant(call, M, N, K, ldb=ld, b_offset=offset) == (TILES, rows, cols, SHIFT), (M, N, K, offset, ld)
    for call, M, N, K, feed, cols in FUSED_CASES:
        assert variant(call, M, N, K) == (FUSED, 16, cols, feed), (call, M, N, K)
    for tile in AT:
        ends = {(K % 128, offset, ld % 4) for _, _, K, offset, ld, *t in LINEAR_TILES if tuple(t) == tile}
        assert {K for K, _, _ in ends} >= {0, 1, 125, 127}
        assert {o for _, o, _ in ends} == {ld for _, _, ld in ends} == {0, 1, 2, 3}


def test_query():
    assert variant(0, 0, 8, 64)[0] == NONE and variant(1, 8, 0, 64)[0] == NONE
    assert variant(0, 9, 8, 15) == (SHORT, 0, 0, 0) and variant(1, 1, 8, 15) == (SHORT, 0, 0, 0)
    assert variant(1, 1, 1536, 7168) == (FUSED, 16, 8, WIDE) and variant(2, 1, 300, 1001) == (FUSED, 16, 8, REGS)
    assert variant(1, 1, 5000, 1004) == (FUSED, 16, 16, DWORD)
    # the quantiser's codes are aligned and padded, a caller's are what they are
    assert variant(1, 2000, 4101, 257)[3] == SHIFT and variant(0, 2000, 4101, 257)[3] == REGS
    assert variant(0, 2000, 4101, 256, a_offset=4)[3] == DWORD and variant(0, 2000, 4101, 256, b_offset=2)[3] == REGS
    f = _lib.load().dsfp8_i8_variant
    v = (ctypes.c_int32 * 4)()
    assert f(0, None, 64, None, 64, 4, 4, 64, None) == -1
    for call, M, N, K in ((3, 4, 4, 64), (-1, 4, 4, 64), (0, -1, 4, 64), (0, 4, 1 << 31, 64), (0, 4, 4, 131072)):
        assert f(call, None, 64, None, 64, M, N, K, v) == -2


# ---- on the GPU -----------------------------------------------------------------------------


def codes(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda", generator=g)


def scales(n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return 0.01 * (0.5 + torch.rand(n, device="cuda", generator=g))


def placed(t, ld, offset, fill):
    """t's rows `ld` elements apart from element `offset` of a buffer full of `fill`; also the buffer."""
    rows, cols = t.shape
    buf = torch.full((offset + rows * ld + 64,), fill, dtype=t.dtype, device=t.device)
    v = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v, buf


def product(a, a_s, b, b_s):
    acc = a.double() @ b.double().t().contiguous()
    return (acc.float() * (a_s[:, None] * b_s[None, :])).bfloat16()


def same(c, want, buf=None, ld=0, offset=0):
    assert torch.equal(c, want), f"{int((c != want).sum())} of {c.numel()} elements differ"
    if buf is not None:
        between = buf[offset:offset + c.shape[0] * ld].view(c.shape[0], ld)[:, c.shape[1]:]
        assert bool((between == 7.0).all()) and bool((buf[:offset] == 7.0).all()), "elements outside were written"


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,feed,rows,cols", GEMM_TILES + GEMM_SPLIT)
def test_gemm(M, N, K, feed, rows, cols):
    import block_scaled_fp8_act_amd as ds
    a, b, a_s, b_s = codes((M, K), 1), codes((N, K), 2), scales(M, 3), scales(N, 4)
    assert variant(0, M, N, K, a_offset=a.data_ptr() % 16, b_offset=b.data_ptr() % 16)[1:] == (rows, cols, feed)
    ld, offset = (N + 3, 5) if K % 2 else (N, 0)    # an output at odd addresses, or contiguous
    c, buf = placed(torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda"), ld, offset, 7.0)
    ds.gemm_i8(a, a_s, b, b_s, out=c)
    same(c, product(a, a_s, b, b_s), buf, ld, offset)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,offset,ld,rows,cols", LINEAR_TILES)
def test_linear_weights_at_any_address(M, N, K, offset, ld, rows, cols):
    """Both linear forms; values around the weight's rows, and in the workspace before the call, that must not count."""
    import block_scaled_fp8_act_amd as ds
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x, u = (torch.randn((M, K), device="cuda", generator=g).bfloat16() for _ in range(2))
    w, buf = placed(codes((N, K), 6), ld, offset, 99)
    w_s = scales(N, 7)
    for call, args, quant in ((1, (x,), ds.row_quant_i8), (2, (x, u), ds.silu_mul_row_quant_i8)):
        assert variant(call, M, N, K, ldb=ld, b_offset=w.data_ptr() % 16) == (TILES, rows, cols, SHIFT)
        work = torch.full((_lib.load().dsfp8_linear_i8_workspace_bytes(M, N, K, call - 1),), 0x5a, dtype=torch.uint8,
                          device="cuda")
        c = (ds.linear_i8 if call == 1 else ds.silu_mul_linear_i8)(*args, w, w_s, workspace=work)
        same(c, product(*quant(*args), w, w_s))
    assert bool((buf[:offset] == 99).all())


@pytest.mark.gpu
@pytest.mark.parametrize("call,M,N,K,feed,cols", FUSED_CASES)
def test_linear_in_one_launch(call, M, N, K, feed, cols):
    import block_scaled_fp8_act_amd as ds
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    x, u = (torch.randn((M, K), device="cuda", generator=g).bfloat16() for _ in range(2))
    w, w_s = codes((N, K), 9), scales(N, 10)
    assert variant(call, M, N, K, b_offset=w.data_ptr() % 16) == (FUSED, 16, cols, feed)
    if call == 1:
        same(ds.linear_i8(x, w, w_s), product(*ds.row_quant_i8(x), w, w_s))
    else:
        same(ds.silu_mul_linear_i8(x, u, w, w_s), product(*ds.silu_mul_row_quant_i8(x, u), w, w_s))
