"""GPU checks of the norms around a residual connection, element by element within the bounds that
oracle/norm.py derives for an fp32 evaluation, plus half a step of each output's type."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as ds
from block_scaled_fp8_act_amd import inputs as I
from oracle import formats as F
from oracle import mxfp4 as MX
from oracle import norm as NM

from gpu_helpers import bf16_to_f64, dev_bf16, host_bits16, host_u8

pytestmark = pytest.mark.gpu

CID = 140


def operands(T, D, seed, post=True, gate="row", residual=True, wtype=torch.bfloat16):
    g = I.rng(CID, seed)
    op = {"x": I.activations((T, D), CID, seed + 1, outlier_frac=0.01)}
    op["residual"] = I.activations((T, D), CID, seed + 2) if residual else None
    op["gate"] = {"none": None, "row": I.to_bf16_bits(g.random((T, D), np.float32)),
                  "channel": I.to_bf16_bits(g.random(D, np.float32))}[gate]
    w = [torch.from_numpy((1 + 0.2 * g.standard_normal(D)).astype(np.float32)).to(wtype) for _ in range(2)]
    return op, w[0], w[1] if post else None


def run(op, w, pw, **kw):
    d = {n: None if v is None else dev_bf16(v) for n, v in op.items()}
    return ds.add_rms_norm(d["x"], w.cuda(), residual=d["residual"], gate=d["gate"],
                           post_weight=None if pw is None else pw.cuda(), **kw)


def expected(op, w, pw, scale=1.0, eps=1e-6):
    v = {n: None if b is None else bf16_to_f64(b) for n, b in op.items()}
    return NM.forward(v["x"], w.double().numpy(), v["residual"], None if pw is None else pw.double().numpy(), v["gate"], scale, eps)


def within(got, ref, bound, half, what):
    err = np.abs(got - ref)
    lim = bound + (np.abs(ref) + bound) * half + 2.0 ** -134
    assert np.all(err <= lim), f"{what}: {float((err / lim).max()):.3f} of the bound"


def check(got, op, w, pw, quant, D, **kw):
    h, dh, y, dy = expected(op, w, pw, **kw)
    got = got if isinstance(got, tuple) else (got,)
    if op["residual"] is not None:
        within(bf16_to_f64(host_bits16(got[-1])), h, dh, 2.0 ** -8, "h")
    if quant is None:
        return within(bf16_to_f64(host_bits16(got[0])), y, dy, 2.0 ** -8, "y")
    block = 32 if quant == "mxfp4" else 128
    T, nb = y.shape[0], -(-D // block)
    top, dtop = (np.pad(v, ((0, 0), (0, nb * block - D))).reshape(T, nb, block).max(axis=2) for v in (np.abs(y), dy))
    if quant == "mxfp4":
        s = host_u8(got[1])
        assert np.all((s == MX.scale_byte(top - dtop)) | (s == MX.scale_byte(top + dtop))), "scales"
        unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), block, axis=1)[:, :D]
        v = MX.values(host_u8(got[0]), s, D)
        a = (np.abs(y) + dy) / unit     # half a step grows with the value
        half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.maximum(1.0, a - 6))) * unit
        assert np.all(np.abs(v - y) <= half + dy), "codes"
        assert not MX.unpack(host_u8(got[0]))[:, D:].any()
    else:
        s = got[1].cpu().numpy().astype(np.float64)
        if quant == "e4m3":
            ref = np.maximum(top, 1e-4) / 448
            assert np.all(np.abs(s - ref) <= dtop / 448 + ref * 2.0 ** -23), "scales"
        else:
            lo, hi = (np.exp2(np.ceil(np.log2(np.maximum(t, 1e-4) / 448))) for t in (top * (1 - 2.0 ** -22) - dtop, top * (1 + 2.0 ** -22) + dtop))
            assert np.all((s == lo) | (s == hi)), "scales"
        sc = np.repeat(s, block, axis=1)[:, :D]
        v = F.e4m3_decode(host_u8(got[0])).astype(np.float64) * sc
        within(v, y, dy + sc * 2.0 ** -10, 2.0 ** -4 + 2.0 ** -22, "codes")


# columns around a chunk of 8, a block of 32 and of 128, and the limits of each kernel
SIZES = [(1, 1), (3, 7), (2, 8), (5, 33), (4, 127), (3, 129), (9, 511), (6, 512), (5, 513), (2, 1000), (3, 2048), (2, 2049),
         (2, 4096), (3, 4100), (2, 7168), (2, 8192), (2, 8193), (1, 16384), (2, 16400), (1, 32769), (1, 65536), (70, 256)]


@pytest.mark.parametrize("quant", [None, "e4m3", "e4m3_ue8m0", "mxfp4"])
@pytest.mark.parametrize("T,D", SIZES)
def test_sandwich(T, D, quant):
    op, w, pw = operands(T, D, 10 * T + D)
    got = run(op, w, pw, scale=0.5, quant=quant)
    check(got, op, w, pw, quant, D, scale=0.5)
    again = run(op, w, pw, scale=0.5, quant=quant)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp4"])
@pytest.mark.parametrize("residual,post,gate,wtype", [(False, False, "none", torch.bfloat16), (True, False, "none", torch.float32),
                                                      (True, True, "none", torch.float32), (True, False, "channel", torch.bfloat16),
                                                      (True, True, "channel", torch.float32), (True, False, "row", torch.bfloat16)])
def test_forms(residual, post, gate, wtype, quant):
    for T, D in [(5, 300), (3, 1537)]:
        op, w, pw = operands(T, D, 77, post, gate, residual, wtype)
        kw = dict(scale=0.22 if residual else 1.0, eps=1e-5)
        check(run(op, w, pw, quant=quant, **kw), op, w, pw, quant, D, **kw)


def test_rows_of_zeros_and_tiny_values():
    """Zeros give zeros (eps keeps the root from zero); values whose squares vanish in fp32 do not disturb it."""
    op, w, pw = operands(4, 200, 5)
    op["x"][0] = 0
    op["residual"][0] = 0
    op["x"][1] = I.to_bf16_bits(np.full(200, 1e-30, np.float32))
    op["residual"][1] = 0
    for quant in (None, "mxfp4"):
        got = run(op, w, pw, quant=quant)
        y = bf16_to_f64(host_bits16(got[0])) if quant is None else MX.values(host_u8(got[0]), host_u8(got[1]), 200)
        assert not y[0].any() and np.isfinite(y).all()
        assert not host_bits16(got[-1])[0].any()
    q, s, _ = run(op, w, pw, quant="e4m3")
    assert np.all(s[0].cpu().numpy() == np.float32(1e-4) / np.float32(448)) and not q[0].any()


def test_squares_past_the_range_give_zeros():
    w = torch.ones(700, dtype=torch.bfloat16, device="cuda")
    x = torch.ones((3, 700), dtype=torch.bfloat16, device="cuda")
    x[1] = 1e25
    y = ds.add_rms_norm(x, w)
    assert not y[1].any() and (y[0] == 1).all() and (y[2] == 1).all()
    q, s = ds.add_rms_norm(x, w, quant="e4m3")
    assert not q[1].any() and torch.isfinite(s).all()
    q, s = ds.add_rms_norm(x, w, quant="mxfp4")
    assert not ds.mxfp4_dequant(q, s, 700)[1].any()


@pytest.mark.parametrize("bad", [0x7fc0, 0x7f80])
def test_nan_and_infinity_stay_in_their_row(bad):
    op, w, pw = operands(5, 700, 6)
    clean = {q: run(op, w, pw, quant=q) for q in (None, "e4m3", "e4m3_ue8m0", "mxfp4")}
    op["x"][2, 699] = bad
    for q, ref in clean.items():
        got = run(op, w, pw, quant=q)
        keep = [0, 1, 3, 4]
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, ref))
        if q is None:
            assert torch.isnan(got[0][2].float()).any()
        elif q == "mxfp4":
            assert (got[1][2] == 255).any()
        else:
            assert not torch.isfinite(got[1][2]).all()


def test_strides_in_place_and_out():
    T, D = 6, 333
    op, w, pw = operands(T, D, 7)
    ref = run(op, w, pw)
    d = {n: dev_bf16(v) for n, v in op.items()}

    def wide(t):
        b = torch.full((T, D + 9), 9.0, dtype=t.dtype, device="cuda")
        b[:, 5:5 + D] = t
        return b
    W = {n: wide(t) for n, t in d.items()}
    v = {n: b[:, 5:5 + D] for n, b in W.items()}
    # h over the residual, y over x
    y, h = ds.add_rms_norm(v["x"], w.cuda(), residual=v["residual"], gate=v["gate"], post_weight=pw.cuda(), out=(v["x"], v["residual"]))
    assert torch.equal(y, ref[0]) and torch.equal(h, ref[1])
    for b in W.values():
        assert (b[:, :5] == 9).all() and (b[:, 5 + D:] == 9).all()
    row_major = torch.full((T, 5), 9.0, device="cuda")
    q, s, h = ds.add_rms_norm(d["x"], w.cuda(), residual=d["residual"], quant="e4m3",
                              out=(None, row_major[:, :3], None))
    q2, s2, h2 = ds.add_rms_norm(d["x"], w.cuda(), residual=d["residual"], quant="e4m3")
    assert torch.equal(q, q2) and torch.equal(s, s2) and (row_major[:, 3:] == 9).all()
    # a gate row for all tokens, given as an expanded matrix or as a vector
    g = d["gate"][0]
    a = ds.add_rms_norm(d["x"], w.cuda(), residual=d["residual"], gate=g)
    b = ds.add_rms_norm(d["x"], w.cuda(), residual=d["residual"], gate=g[None].expand(T, D))
    c = ds.add_rms_norm(d["x"], w.cuda(), residual=d["residual"], gate=g[None].expand(T, D).contiguous())
    assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(a, b, c))


def test_no_rows():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    assert ds.add_rms_norm(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 64)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("quant,shapes", [(None, [(0, 300)]), ("e4m3", [(0, 300), (0, 3)]), ("e4m3_ue8m0", [(0, 300), (0, 3)]),
                                          ("mxfp4", [(0, 160), (0, 10)])])
def test_no_rows_of_any_output(quant, shapes, residual):
    w = torch.ones(300, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 300), dtype=torch.bfloat16, device="cuda")
    got = ds.add_rms_norm(x, w, residual=x if residual else None, quant=quant)
    got = got if isinstance(got, tuple) else (got,)
    assert [tuple(t.shape) for t in got] == shapes + ([(0, 300)] if residual else [])


@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp4"])
def test_more_rows_than_one_launch_takes(quant):
    """2^21 + 9 rows go in two launches; the rows around the cut as in a call of their own."""
    T, D = 2 ** 21 + 9, 16
    x = torch.randn((T, D), device="cuda").bfloat16()
    r = torch.randn((T, D), device="cuda").bfloat16()
    g = torch.rand((T, D), device="cuda").bfloat16()
    w = torch.randn(D, device="cuda")
    for gate in (g, g[0]):
        whole = ds.add_rms_norm(x, w, residual=r, gate=gate, scale=0.5, quant=quant)
        cut = slice(2 ** 21 - 5, T)
        part = ds.add_rms_norm(x[cut], w, residual=r[cut], gate=gate if gate.dim() == 1 else gate[cut], scale=0.5, quant=quant)
        assert all(torch.equal(a[cut], b) for a, b in zip(whole, part))


@pytest.mark.parametrize("D", [520, 4000, 7168, 16000, 33000])
@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp4"])
def test_a_row_does_not_depend_on_the_number_of_rows(D, quant):
    op, w, pw = operands(4, D, 9)
    op = {n: v if v is None else np.tile(v, (400, 1)) for n, v in op.items()}
    whole = run(op, w, pw, scale=0.5, quant=quant)
    few = run({n: v if v is None else v[:4] for n, v in op.items()}, w, pw, scale=0.5, quant=quant)
    for a, b in zip(whole, few):
        assert torch.equal(a[:4], b) and torch.equal(a[-4:], b)


def test_graph():
    T, D = 40, 2304
    op, w, pw = operands(T, D, 8)
    d = {n: dev_bf16(v) for n, v in op.items()}
    wd, pd = w.cuda(), pw.cuda()
    stream = d["residual"].clone()
    q, s = ds.mxfp4_empty(T, D, "cuda")

    def step():                     # the residual stream updated in place
        ds.add_rms_norm(d["x"], wd, residual=stream, post_weight=pd, gate=d["gate"], quant="mxfp4", out=(q, s, stream))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(4):
        d["x"].copy_(dev_bf16(I.activations((T, D), CID, 20 + seed)))
        before = stream.clone()
        g.replay()
        torch.cuda.synchronize()
        got = q.clone(), s.clone(), stream.clone()
        stream.copy_(before)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], q) and torch.equal(got[1], s) and torch.equal(got[2], stream)


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: ds.add_rms_norm(x, w, gate=x), lambda: ds.add_rms_norm(x, w, post_weight=w), lambda: ds.add_rms_norm(x, w, scale=2.0),
                lambda: ds.add_rms_norm(x, w[:63]), lambda: ds.add_rms_norm(x, w.half()), lambda: ds.add_rms_norm(x.float(), w),
                lambda: ds.add_rms_norm(x, w, residual=x[:3]), lambda: ds.add_rms_norm(x, w, residual=x, post_weight=w.float()),
                lambda: ds.add_rms_norm(x, w, residual=x, gate=w[:5]), lambda: ds.add_rms_norm(x, w, quant="int8"),
                lambda: ds.add_rms_norm(x, w, eps=-1.0), lambda: ds.add_rms_norm(x.t(), w[:4]), lambda: ds.add_rms_norm(x.cpu(), w),
                lambda: ds.add_rms_norm(x, w.cpu()), lambda: ds.add_rms_norm(x, w, residual=x, out=(x,)),
                lambda: ds.add_rms_norm(torch.zeros((1, 65537), dtype=torch.bfloat16, device="cuda"),
                                        torch.zeros(65537, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ds.Dsfp8Error):
            bad()


@pytest.mark.parametrize("quant", ["e4m3", "e4m3_ue8m0", "mxfp4"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("given", [(True, False), (False, True), (True, True)])
def test_some_outputs_given(quant, residual, given):
    """Whichever of y, s and h the caller supplies is what is written and returned."""
    T, D = 7, 333
    op, w, _ = operands(T, D, 11, post=False, gate="none", residual=residual)
    ref = run(op, w, None, quant=quant)
    buf = list(ds.mxfp4_empty(T, D, "cuda")) if quant == "mxfp4" else [
        torch.empty((T, D), dtype=torch.uint8, device="cuda"), torch.empty((T, 3), device="cuda")]
    for b in buf:
        b.fill_(9)
    out = [b if g else None for b, g in zip(buf, given)]
    h = [torch.empty((T, D), dtype=torch.bfloat16, device="cuda")] if residual else []
    got = run(op, w, None, quant=quant, out=(*out, *h))
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    for g, b in zip(got, [*out, *h]):
        assert b is None or (g.data_ptr() == b.data_ptr() and g.stride() == b.stride())


# each number of threads and chunks that fp32 weights of more than 2048 columns take, for few rows and, where that
# is another kernel, for more than two a CU
@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp4"])
@pytest.mark.parametrize("T,D", [(3, 2051), (3, 4100), (3, 7171), (3, 16003), (2, 20001), (2, 33001), (1, 65529), (600, 2051),
                                 (600, 4100), (530, 7171), (520, 16003)])
def test_wide_rows_with_fp32_weights(T, D, quant):
    assert T < 4 or T > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    # the sandwich for a few rows, many times over where there are more: the oracle's time is that of seven
    n = min(T, 7)
    op, w, pw = operands(n, D, 13 + D, wtype=torch.float32)
    many = {k: v if v is None else np.resize(v, (T, D)) for k, v in op.items()}
    got = run(many, w, pw, scale=0.5, quant=quant)
    for r in range(0, T - n + 1, max(1, (T - n) // 3)):
        r -= r % n
        check(tuple(t[r:r + n] for t in got), op, w, pw, quant, D, scale=0.5)


@pytest.mark.parametrize("T,D", [(5, 100), (600, 128), (7, 300), (700, 513), (5, 2100), (530, 2100), (3, 4000), (9, 7168), (520, 7001),
                                 (2, 16000), (2, 20000), (2, 40000)])
def test_e4m3_codes_of_halfway_cases(T, D):
    """Without a residual and with bf16 weights a code is that of the exact quotient, halfway cases included, and a row's
    codes do not change with a power of two."""
    x, w = NM.halfway_rows(T, D, I.rng(CID, 60 + D))
    want = NM.e4m3_codes(x, w)
    x[1::3] *= 2.0 ** -5
    x[2::3] *= 2.0 ** 20
    q, s = ds.add_rms_norm(torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(w).bfloat16().cuda(), eps=0.0, quant="e4m3")
    assert (s > 1e-4 / 448).all()
    assert np.array_equal(host_u8(q), want)


def test_eps_zero():
    """eps = 0 is taken: a row of zeros, or of values whose squares vanish in fp32, shows it and changes no other row."""
    x = torch.ones((5, 300), dtype=torch.bfloat16, device="cuda")
    x[1], x[3] = 0, 1e-30
    w = torch.ones(300, device="cuda")
    y = ds.add_rms_norm(x, w, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isinf(y[3]).all() and (y[[0, 2, 4]] == 1).all()
    for quant in ("e4m3", "e4m3_ue8m0", "mxfp4"):
        q, s = ds.add_rms_norm(x, w, eps=0.0, quant=quant)
        shown = s == 255 if quant == "mxfp4" else ~torch.isfinite(s)
        assert shown[[1, 3]].all() and not shown[[0, 2, 4]].any()
    y, h = ds.add_rms_norm(x, w, residual=x, post_weight=w, eps=0.0)
    assert torch.isnan(h[1]).all() and torch.isinf(h[3]).all() and (h[[0, 2, 4]] == 2).all() and (y[[0, 2, 4]] == 1).all()
