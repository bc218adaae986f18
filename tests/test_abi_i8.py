"""Refusals of the int8 and few-token entry points, provoked on the host with fake
pointers (no kernel launch; only calls that are rejected or empty are made)."""

import os

import pytest

from block_scaled_fp8_act_amd import _lib

OK, NULL, SHAPE, LD, ALIGN, FMT, WS, LAUNCH, DTYPE = 0, -1, -2, -3, -4, -5, -6, -7, -8
P = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from block_scaled_fp8_act_amd import build
        build.build()
    return _lib.load()


def test_row_quant(lib):
    f = lib.dsfp8_row_quant_i8      # x, dtype, M, K, ldx, y, ldy, s, stream
    assert f(P, 2, 4, 32, 32, P, 32, P, None) == DTYPE
    assert f(P, 1, -1, 32, 32, P, 32, P, None) == SHAPE
    assert f(P, 1, 4, 1 << 31, 1 << 31, P, 1 << 31, P, None) == SHAPE
    assert f(None, 1, 4, 32, 32, P, 32, P, None) == NULL
    assert f(P, 1, 4, 32, 32, None, 32, P, None) == NULL
    assert f(P, 1, 4, 32, 32, P, 32, None, None) == NULL
    assert f(P, 1, 4, 32, 31, P, 32, P, None) == LD
    assert f(P, 1, 4, 32, 32, P, 31, P, None) == LD
    assert f(P + 1, 1, 4, 32, 32, P, 32, P, None) == ALIGN
    assert f(P + 2, 0, 4, 32, 32, P, 32, P, None) == ALIGN
    assert f(P, 1, 4, 32, 32, P, 32, P + 2, None) == ALIGN
    assert f(None, 1, 0, 32, 32, None, 32, None, None) == OK
    g = lib.dsfp8_silu_mul_row_quant_i8     # g, ldg, u, ldu, M, I, y, ldy, s, stream
    assert g(P, 32, None, 32, 4, 32, P, 32, P, None) == NULL
    assert g(P, 32, P, 31, 4, 32, P, 32, P, None) == LD
    assert g(P, 32, P + 1, 32, 4, 32, P, 32, P, None) == ALIGN
    assert g(None, 32, None, 32, 0, 32, None, 32, None, None) == OK


def test_gemm(lib):
    f = lib.dsfp8_gemm_i8           # A, lda, a_s, B, ldb, b_s, C, ldc, M, N, K, stream
    assert f(P, 64, P, P, 64, P, P, 8, 4, 8, 131072, None) == SHAPE
    assert f(P, 64, P, P, 64, P, P, 8, 4, 8, -1, None) == SHAPE
    assert f(P, 64, P, P, 64, P, P, 8, -4, 8, 64, None) == SHAPE
    assert f(P, 64, P, P, 64, P, P, 1 << 31, 4, 1 << 31, 64, None) == SHAPE
    for i, want in [(0, NULL), (2, NULL), (3, NULL), (5, NULL), (6, NULL)]:
        a = [P, 64, P, P, 64, P, P, 8, 4, 8, 64, None]
        a[i] = None
        assert f(*a) == want
    for i in (1, 4, 7):
        a = [P, 64, P, P, 64, P, P, 8, 4, 8, 64, None]
        a[i] -= 1
        assert f(*a) == LD
    for i, off in [(2, 1), (5, 2), (6, 1)]:
        a = [P, 64, P, P, 64, P, P, 8, 4, 8, 64, None]
        a[i] += off
        assert f(*a) == ALIGN
    assert f(None, 64, None, P, 64, P, None, 8, 0, 8, 64, None) == OK
    assert f(P, 64, P, None, 64, None, None, 8, 4, 0, 64, None) == OK


def test_linear(lib):
    bytes_ = lib.dsfp8_linear_i8_workspace_bytes        # M, N, K, gated
    need = bytes_(40, 8, 50, 0)
    assert need == 40 * 64 + 160
    assert bytes_(-1, 8, 50, 0) == 0 and bytes_(4, -8, 50, 0) == 0 and bytes_(4, 8, 131072, 0) == 0
    assert bytes_(4, 8, 50, 0) == 0 and bytes_(4, 8, 50, 1) == 0    # one launch: no scratch
    assert bytes_(16, 8, 1040, 0) == 16 * 1044
    assert bytes_(4, 8, 8, 0) == 4 * 16 + 16
    f = lib.dsfp8_linear_i8         # x, ldx, B, ldb, b_s, C, ldc, M, N, K, ws, wsb, stream
    ok = [P, 50, P, 50, P, P, 8, 40, 8, 50, P, need, None]

    def with_(i, v, *more):
        a = list(ok)
        for j, w in ((i, v),) + more:
            a[j] = w
        return f(*a)

    assert with_(0, None) == NULL and with_(2, None) == NULL and with_(4, None) == NULL and with_(5, None) == NULL
    assert with_(10, None) == NULL and with_(10, P + 8) == ALIGN and with_(11, need - 1) == WS
    assert with_(0, P + 1) == ALIGN and with_(4, P + 2) == ALIGN and with_(5, P + 1) == ALIGN
    assert with_(1, 49) == LD and with_(3, 49) == LD and with_(6, 7) == LD
    assert with_(7, -1) == SHAPE and with_(8, -1) == SHAPE and with_(9, 131072) == SHAPE
    # few rows: no workspace, the other arguments as ever
    few = ((7, 4), (10, None), (11, 0))
    assert with_(0, None, *few) == NULL and with_(2, None, *few) == NULL and with_(5, None, *few) == NULL
    assert with_(1, 49, *few) == LD and with_(6, 7, *few) == LD and with_(5, P + 1, *few) == ALIGN
    assert f(None, 50, P, 50, P, None, 8, 0, 8, 50, None, 0, None) == OK
    g = lib.dsfp8_silu_mul_linear_i8    # g, ldg, u, ldu, B, ldb, b_s, C, ldc, M, N, K, ws, wsb, stream
    assert g(P, 50, None, 50, P, 50, P, P, 8, 40, 8, 50, P, need, None) == NULL
    assert g(P, 50, P, 49, P, 50, P, P, 8, 40, 8, 50, P, need, None) == LD
    assert g(P, 50, P + 1, 50, P, 50, P, P, 8, 40, 8, 50, P, need, None) == ALIGN


def test_moe_few(lib):
    T, k, E, D, F = 3, 2, 4, 256, 128
    need = lib.dsfp8_moe_few_workspace_bytes(T, k, F)
    assert need > 0
    for bad in [(65, k, F), (-1, k, F), (T, 0, F), (T, 17, F), (T, k, -1)]:
        assert lib.dsfp8_moe_few_workspace_bytes(*bad) == 0
    # x, ldx, W13, ld, s13, ld, W2, ld, s2, ld, fmt, idx, ldi, wt, ldwt, T, k, E, D, F, out, ldo, ws, wsb, stream
    ok = [P, D, P, D, P, 2, P, F, P, 1, 0, P, k, P, k, T, k, E, D, F, P, D, P, need, None]

    def with_(*changes, base=ok):
        a = list(base)
        for i, v in changes:
            a[i] = v
        return lib.dsfp8_moe_few(*a)

    assert with_((10, 2)) == DTYPE and with_((10, -1)) == DTYPE
    assert with_((15, 65), (23, 1 << 30)) == SHAPE and with_((15, -1)) == SHAPE
    assert with_((16, 0)) == SHAPE and with_((16, 17)) == SHAPE
    assert with_((17, 0)) == SHAPE and with_((17, 4097)) == SHAPE
    assert with_((18, -1)) == SHAPE and with_((19, 1 << 30)) == SHAPE
    assert with_((18, (1 << 26) + 1)) == SHAPE and with_((19, (1 << 26) + 1)) == SHAPE
    assert lib.dsfp8_moe_few_workspace_bytes(T, k, (1 << 26) + 1) == 0
    for i in (0, 2, 4, 6, 8, 11, 13, 20, 22):
        assert with_((i, None)) == NULL, i
    for i in (1, 3, 5, 7, 9, 12, 14, 21):
        assert with_((i, ok[i] - 1)) == LD, i
    # int8: scales are one row per expert
    assert with_((10, 1)) == LD and with_((10, 1), (5, 2 * F)) == LD and with_((10, 1), (5, 2 * F), (9, D), (23, 0)) == WS
    for i, off in [(0, 1), (4, 2), (8, 1), (11, 2), (13, 1), (20, 1), (22, 8)]:
        assert with_((i, P + off)) == ALIGN, i
    assert with_((23, need - 1)) == WS
    assert with_((15, 0), (0, None), (11, None), (13, None), (20, None), (22, None), (23, 0)) == OK
    assert with_((18, 0), (1, 0), (3, 0), (5, 0), (21, 0)) == OK
