"""Refusals of the MXFP4, gate and norm entry points, provoked on the host with fake pointers (no
kernel launch; only calls that are rejected or empty are made)."""

import os

import pytest

from block_scaled_fp8_act_amd import _lib

OK, NULL, SHAPE, LD, ALIGN, WS, DTYPE, UNSUP, SCORE = 0, -1, -2, -3, -4, -6, -8, -9, -11
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from block_scaled_fp8_act_amd import build
        build.build()
    return _lib.load()


def caller(fn, **args):
    names = list(args)

    def call(**kw):
        assert set(kw) <= set(names), kw
        return fn(*[kw.get(n, args[n]) for n in names])
    return call


def test_quant(lib):
    c = caller(lib.dsfp8_mxfp4_quant, x=P, dtype=1, M=4, K=50, ldx=50, y=P, ldy=32, s=P, lds=16, stream=None)
    assert c(dtype=2) == DTYPE
    assert c(M=-1) == SHAPE and c(K=-1) == SHAPE and c(M=1 << 31) == SHAPE and c(K=1 << 31, ldx=1 << 31) == SHAPE
    assert c(x=None) == NULL and c(y=None) == NULL and c(s=None) == NULL
    assert c(ldx=49) == LD and c(ldy=16) == LD and c(ldy=40) == LD and c(lds=0) == LD and c(lds=24) == LD
    assert c(K=513, ldx=513, ldy=272) == LD                 # 17 blocks: 32 bytes of scales
    assert c(x=P + 1) == ALIGN and c(x=P + 2, dtype=0) == ALIGN and c(y=P + 8) == ALIGN and c(s=P + 4) == ALIGN
    assert c(M=0, x=None, y=None, s=None) == OK and c(K=0, ldy=0, lds=0, x=None, y=None, s=None) == OK
    c = caller(lib.dsfp8_silu_mul_mxfp4_quant, g=P, ldg=50, u=P, ldu=50, M=4, I=50, y=P, ldy=32, s=P, lds=16, stream=None)
    assert c(M=-1) == SHAPE and c(g=None) == NULL and c(u=None) == NULL and c(ldg=49) == LD and c(ldu=49) == LD
    assert c(u=P + 1) == ALIGN and c(lds=8) == LD and c(M=0, g=None, u=None, y=None, s=None) == OK
    c = caller(lib.dsfp8_mxfp4_dequant, q=P, ldq=32, s=P, lds=16, M=4, K=50, out=P, ldo=50, stream=None)
    assert c(M=-1) == SHAPE and c(q=None) == NULL and c(s=None) == NULL and c(out=None) == NULL
    assert c(ldq=16) == LD and c(lds=8) == LD and c(ldo=49) == LD
    assert c(q=P + 4) == ALIGN and c(s=P + 1) == ALIGN and c(out=P + 1) == ALIGN
    assert c(M=0, q=None, s=None, out=None) == OK


def test_gemm(lib):
    c = caller(lib.dsfp8_gemm_mxfp4, A=P, lda=32, a_s=P, ldas=16, B=P, ldb=32, b_s=P, ldbs=16, C=P, ldc=8, M=4, N=8, K=64,
               stream=None)
    for n in ("M", "N", "K"):
        assert c(**{n: -1}) == SHAPE
    assert c(N=1 << 31, ldc=1 << 31) == SHAPE
    for n in ("A", "a_s", "B", "b_s", "C"):
        assert c(**{n: None}) == NULL
    for n in ("lda", "ldb"):
        assert c(**{n: 16}) == LD and c(**{n: 40}) == LD and c(**{n: 1 << 23}) == UNSUP
    for n in ("ldas", "ldbs"):
        assert c(**{n: 0}) == LD and c(**{n: 24}) == LD and c(**{n: 1 << 23}) == UNSUP
    assert c(ldc=7) == LD
    for n in ("A", "a_s", "B", "b_s"):
        assert c(**{n: P + 8}) == ALIGN
    assert c(C=P + 1) == ALIGN
    assert c(M=0, A=None, a_s=None, C=None) == OK and c(N=0, B=None, b_s=None, C=None) == OK


def test_linear(lib):
    need = lib.dsfp8_linear_mxfp4_workspace_bytes
    assert need(400, 8, 50) == 400 * 48
    assert need(-1, 8, 50) == 0 and need(4, -8, 50) == 0 and need(4, 8, 1 << 24) == 0
    c = caller(lib.dsfp8_linear_mxfp4, x=P, ldx=50, B=P, ldb=32, b_s=P, ldbs=16, C=P, ldc=8, M=400, N=8, K=50, ws=P,
               wsb=400 * 48, stream=None)
    assert c(M=-1) == SHAPE and c(N=-1) == SHAPE and c(K=-1) == SHAPE
    for n in ("x", "B", "b_s", "C", "ws"):
        assert c(**{n: None}) == NULL
    assert c(wsb=400 * 48 - 1) == WS and c(ws=P + 8) == ALIGN
    assert c(ldx=49) == LD and c(ldb=16) == LD and c(ldbs=8) == LD and c(ldc=7) == LD
    assert c(x=P + 1) == ALIGN and c(B=P + 1) == ALIGN and c(b_s=P + 1) == ALIGN and c(C=P + 1) == ALIGN
    assert c(ldb=1 << 23) == UNSUP
    assert c(M=0, x=None, C=None, ws=None, wsb=0) == OK and c(N=0, B=None, b_s=None, C=None) == OK


def test_linear_past_its_limit(lib):
    """K from 2^24 - 31 on, whose rows of codes the product does not take: UNSUPPORTED, with the workspace that the
    query asks for (none) and with any other."""
    c = caller(lib.dsfp8_linear_mxfp4, x=P, ldx=1 << 25, B=P, ldb=1 << 23, b_s=P, ldbs=1 << 19, C=P, ldc=8, M=4, N=8,
               K=1 << 24, ws=None, wsb=0, stream=None)
    for M in (1, 4, 400):
        for K in ((1 << 24) - 31, 1 << 24, (1 << 24) + 5):
            assert lib.dsfp8_linear_mxfp4_workspace_bytes(M, 8, K) == 0
            assert c(M=M, K=K) == UNSUP and c(M=M, K=K, ws=P, wsb=1 << 40) == UNSUP and c(M=M, K=K, ws=P, wsb=16) == UNSUP
        assert lib.dsfp8_linear_mxfp4_workspace_bytes(M, 8, (1 << 24) - 32) > 0
        assert c(M=M, K=(1 << 24) - 32, ldb=(1 << 23) - 16) == WS


def test_grouped(lib):
    c = caller(lib.dsfp8_grouped_gemm_mxfp4, A=P, a_rows=10, lda=32, a_s=P, ldas=16, rows=None, B=P, ldb=32, b_s=P,
               ldbs=16, offsets=P, E=3, M=10, N=8, K=64, C=P, ldc=8, stream=None)
    assert c(E=0) == SHAPE and c(E=65537) == SHAPE and c(M=-1) == SHAPE and c(a_rows=-1) == SHAPE
    assert c(a_rows=9) == SHAPE and c(a_rows=0, rows=P) == SHAPE
    assert c(offsets=None) == NULL and c(A=None) == NULL and c(B=None) == NULL and c(C=None) == NULL
    assert c(offsets=P + 2) == ALIGN and c(rows=P + 2) == ALIGN and c(a_s=P + 4) == ALIGN
    assert c(lda=16) == LD and c(ldbs=8) == LD and c(ldc=7) == LD
    assert c(rows=P, a_rows=1 << 20, lda=1 << 11) == UNSUP
    assert c(M=0) == OK and c(N=0) == OK


def test_variant(lib):
    import ctypes
    v = (ctypes.c_int32 * 2)()
    c = caller(lib.dsfp8_mxfp4_variant, E=0, M=4, N=8, K=64, v=ctypes.addressof(v))
    assert c(v=None) == NULL and c(E=-1) == SHAPE and c(E=65537) == SHAPE
    assert c(M=-1) == SHAPE and c(N=-1) == SHAPE and c(K=-1) == SHAPE
    assert c() == OK and tuple(v) == (16, 16)
    assert c(M=0) == OK and tuple(v) == (0, 0)
    # more tiles of 16 rows than one launch holds threads for
    assert c(M=1, N=(1 << 31) - 1, K=32) == OK and v[0] > 32
    assert lib.dsfp8_linear_mxfp4_workspace_bytes(1, (1 << 31) - 1, 32) > 0


def test_gate(lib):
    c = caller(lib.dsfp8_moe_gate, logits=P, dtype=0, ldl=64, bias=None, T=4, E=64, k=8, groups=8, top=4, score=0, renorm=1,
               scale=1.0, indices=P, ldi=8, weights=P, ldw=8, stream=None)
    assert c(dtype=2) == DTYPE and c(score=2) == SCORE
    assert c(T=-1) == SHAPE and c(T=1 << 26) == SHAPE and c(E=0) == SHAPE and c(E=4097, ldl=4097, groups=1, top=1) == SHAPE
    assert c(k=0) == SHAPE and c(k=17, ldi=17, ldw=17) == SHAPE and c(groups=0) == SHAPE and c(groups=7) == SHAPE
    assert c(E=128, ldl=128, groups=128) == SHAPE and c(top=0) == SHAPE and c(top=9) == SHAPE
    assert c(top=1, k=9, ldi=9, ldw=9) == SHAPE             # 8 experts in the groups kept
    assert c(logits=None) == NULL and c(indices=None) == NULL and c(weights=None) == NULL
    assert c(ldl=63) == LD and c(ldi=7) == LD and c(ldw=7) == LD
    assert c(logits=P + 2) == ALIGN and c(bias=P + 2) == ALIGN and c(indices=P + 2) == ALIGN and c(weights=P + 1) == ALIGN
    assert c(T=0, logits=None, indices=None, weights=None) == OK
    assert "score" in lib.dsfp8_status_string(SCORE).decode()


def test_norm(lib):
    c = caller(lib.dsfp8_add_rms_norm, x=P, ldx=50, residual=P, ldr=50, gate=P, ldg=50, post=P, w=P, wd=1, scale=1.0,
               eps=1e-6, T=4, D=50, h=P, ldh=50, y=P, ldy=50, fmt=0, s=None, srs=0, sks=0, stream=None)
    assert c(wd=2) == DTYPE and c(fmt=4) == DTYPE and c(fmt=-1) == DTYPE
    assert c(T=-1) == SHAPE and c(D=-1) == SHAPE and c(D=65537, ldx=1 << 17) == SHAPE and c(eps=-1.0) == SHAPE
    assert c(eps=float("nan")) == SHAPE
    assert c(residual=None) == SHAPE and c(residual=None, post=None) == SHAPE
    assert c(residual=None, post=None, gate=None, scale=0.5) == SHAPE
    for n in ("x", "w", "h", "y"):
        assert c(**{n: None}) == NULL
    for n in ("ldx", "ldr", "ldg", "ldh", "ldy"):
        assert c(**{n: 49}) == LD
    for n in ("x", "residual", "gate", "post", "w", "h", "y"):
        assert c(**{n: P + 1}) == ALIGN
    assert c(w=P + 2, wd=0) == ALIGN and c(post=P + 2, wd=0) == ALIGN
    assert c(fmt=1, srs=1, sks=4) == NULL and c(fmt=1, s=P + 2, srs=1, sks=4) == ALIGN
    assert c(fmt=2, ldy=49, s=P, srs=1, sks=4) == LD and c(fmt=1, s=P, srs=0, sks=4) == LD
    assert c(fmt=3, ldy=40, s=P, srs=16) == LD and c(fmt=3, ldy=32, s=P, srs=8) == LD
    assert c(fmt=3, ldy=32, s=P + 8, srs=16) == ALIGN and c(fmt=3, ldy=32, s=None, srs=16) == NULL
    assert c(T=0, x=None, residual=None, post=None, gate=None, w=None, h=None, y=None) == OK
