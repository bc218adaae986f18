"""dsfp8: block-scaled FP8 linear layer for AMD MI355X (gfx950).

Python binding of libdsfp8.so.  Each function checks tensor placement and
dtypes, allocates its outputs with torch on the input's device, and calls the
C entry point of the same name on torch's current stream; every step of the
computation runs in the library's HIP kernels.  e4m3 tensors are exchanged as
``torch.uint8`` (``torch.float8_e4m3fn`` inputs are accepted and viewed as
bytes).  Scales are ``torch.float32``.  Activation scales are indexed
``[M, ceil(K/128)]`` as on the pages; the quantisers return them stored
K-block-major (a transposed view, strides ``(1, M)``), which is the layout the
products read fastest, and the products accept either storage order.

The operations follow the DeepSeek-V3 inference kernels as described in the
"DeepSeek-V3 Administrator & Developer Guide" (sections 6.3, 6.4, 8.5) and the
DocSearch index of the DeepSeek-V3 README (item 3, weight_scale_inv); see
include/dsfp8.h for the exact contracts.

int8 tensors are ``torch.int8`` with one fp32 scale per row (a token of an
activation, an output channel of a weight).  The workspaces that the calls
below allocate with torch may be passed in instead (``workspace=``, of at least
the bytes that the calls' ``*_workspace_bytes`` say), so that a serving loop
allocates nothing.
"""

import torch

from . import _lib

BLOCK = 128
_SCALE_FMT = {"fp32": 0, "ue8m0": 1}


class Dsfp8Error(ValueError):
    """A libdsfp8 call rejected its arguments or failed to launch."""


def kblocks(n):
    return (int(n) + BLOCK - 1) // BLOCK


def status_string(st):
    return _lib.load().dsfp8_status_string(int(st)).decode()


def abi_version():
    return _lib.load().dsfp8_abi_version()


def _check(name, st):
    if st != 0:
        raise Dsfp8Error(f"{name}: {status_string(st)} (status {st})")


def _fmt(scale_fmt):
    if scale_fmt not in _SCALE_FMT:
        raise Dsfp8Error(f"scale_fmt must be one of {sorted(_SCALE_FMT)}, got {scale_fmt!r}")
    return _SCALE_FMT[scale_fmt]


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _mat(t, name, dtypes, dim=2):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise Dsfp8Error(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise Dsfp8Error(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.dim() != dim:
        raise Dsfp8Error(f"{name} must be {dim}-D, got {t.dim()} dimensions")
    if t.numel() > 0 and t.stride(-1) != 1 and not t.is_contiguous():
        raise Dsfp8Error(f"{name}: the last dimension needs stride 1")
    return t


def _ld(t):
    """Row stride; a contiguous tensor's own says nothing where it has a single row."""
    return t.shape[-1] if t.is_contiguous() or t.numel() == 0 else t.stride(-2)


def _scale_strides(t):
    """(row stride, K-block stride) of an activation-scale matrix [M, KB]."""
    M, KB = t.shape
    rs = t.stride(0) if M > 1 else (1 if KB <= 1 or t.stride(1) != 1 else KB)
    ks = t.stride(1) if KB > 1 else (1 if M <= 1 or t.stride(0) != 1 else M)
    return rs, ks


def _scale_matrix(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or t.dim() != 2:
        raise Dsfp8Error(f"{name} must be a 2-D float32 CUDA tensor")
    return _scale_strides(t)


def new_scales(M, KB, device):
    """An activation-scale matrix [M, KB] stored K-block-major (strides (1, M))."""
    return torch.empty((KB, M), dtype=torch.float32, device=device).t()


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _out(out, shape, dtype, device, name):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _mat(_bytes(out), name, (dtype,), dim=len(shape))
    if tuple(out.shape) != tuple(shape) or out.device != device:
        raise Dsfp8Error(f"{name} must be {tuple(shape)} on {device}, got {tuple(out.shape)} on {out.device}")
    return _bytes(out)


def _scales_out(out, M, KB, device):
    if out is None:
        return new_scales(M, KB, device)
    if tuple(out.shape) != (M, KB) or out.device != device:
        raise Dsfp8Error(f"s must be {(M, KB)} on {device}, got {tuple(out.shape)} on {out.device}")
    _scale_matrix(out, "s")
    return out


def act_quant(x, scale_fmt="fp32", out=None):
    """Quantise bf16 ``x [M, K]`` per row and per 128 columns.

    Returns ``(y uint8 [M, K], s float32 [M, ceil(K/128)])`` with x ~= e4m3(y) * s.
    ``out`` may supply preallocated ``(y, s)`` (row strides are honoured; s
    may be row-major or K-block-major).
    """
    _mat(x, "x", (torch.bfloat16,))
    M, K = x.shape
    yo, so = out if out is not None else (None, None)
    y = _out(yo, (M, K), torch.uint8, x.device, "y")
    s = _scales_out(so, M, kblocks(K), x.device)
    srs, sks = _scale_strides(s)
    st = _lib.load().dsfp8_act_quant(x.data_ptr(), M, K, _ld(x), y.data_ptr(), _ld(y), s.data_ptr(), srs, sks,
                                     _fmt(scale_fmt), _stream(x))
    _check("act_quant", st)
    return y, s


def silu_mul_act_quant(g, u, scale_fmt="fp32", return_h=False, out=None):
    """``act_quant(bf16(SiLU(g) * u))`` in one pass; optionally also return h.

    ``out`` may supply preallocated ``(y, s)``."""
    _mat(g, "g", (torch.bfloat16,))
    _mat(u, "u", (torch.bfloat16,))
    if g.shape != u.shape:
        raise Dsfp8Error(f"g and u must have the same shape, got {tuple(g.shape)} and {tuple(u.shape)}")
    M, I = g.shape
    yo, so = out if out is not None else (None, None)
    y = _out(yo, (M, I), torch.uint8, g.device, "y")
    s = _scales_out(so, M, kblocks(I), g.device)
    srs, sks = _scale_strides(s)
    h = torch.empty((M, I), dtype=torch.bfloat16, device=g.device) if return_h else None
    st = _lib.load().dsfp8_silu_mul_act_quant(
        g.data_ptr(), _ld(g), u.data_ptr(), _ld(u), M, I, y.data_ptr(), _ld(y), s.data_ptr(), srs, sks,
        h.data_ptr() if h is not None else None, I, _fmt(scale_fmt), _stream(g))
    _check("silu_mul_act_quant", st)
    return (y, s, h) if return_h else (y, s)


def weight_quant(w, scale_fmt="fp32"):
    """Quantise fp32 or bf16 weights ``[N, K]`` to e4m3 with 128x128 fp32 block scales."""
    _mat(w, "w", (torch.float32, torch.bfloat16))
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    S = torch.empty((kblocks(N), kblocks(K)), dtype=torch.float32, device=w.device)
    dtype = 0 if w.dtype == torch.float32 else 1
    st = _lib.load().dsfp8_weight_quant(w.data_ptr(), dtype, N, K, _ld(w), q.data_ptr(), K, S.data_ptr(),
                                        kblocks(K), _fmt(scale_fmt), _stream(w))
    _check("weight_quant", st)
    return q, S


def weight_dequant(q, S, out=None):
    """bf16 ``[N, K]`` = e4m3 ``q`` times its 128x128 block scale ``S``."""
    q = _mat(_bytes(q), "w", (torch.uint8,))
    _mat(S, "s", (torch.float32,))
    N, K = q.shape
    if tuple(S.shape) != (kblocks(N), kblocks(K)):
        raise Dsfp8Error(f"scale grid must be {(kblocks(N), kblocks(K))}, got {tuple(S.shape)}")
    out = _out(out, (N, K), torch.bfloat16, q.device, "out")
    st = _lib.load().dsfp8_weight_dequant(q.data_ptr(), N, K, _ld(q), S.data_ptr(), _ld(S), out.data_ptr(),
                                          _ld(out), _stream(q))
    _check("weight_dequant", st)
    return out


def gemm(a, a_s, b, b_s, out=None, scale_fmt="fp32"):
    """bf16 ``C [M, N] = A W^T`` with per-K-block scales (A e4m3 [M,K], W e4m3 [N,K]).

    ``scale_fmt="ue8m0"`` declares every scale a power of two (as produced by
    the quantisers with that format); the matrix instruction then applies
    them from their exponents.
    """
    a = _mat(_bytes(a), "a", (torch.uint8,))
    b = _mat(_bytes(b), "b", (torch.uint8,))
    ars, aks = _scale_matrix(a_s, "a_s")
    _mat(b_s, "b_s", (torch.float32,))
    M, K = a.shape
    N, K2 = b.shape
    if K2 != K:
        raise Dsfp8Error(f"a and b disagree on K: {K} vs {K2}")
    if tuple(a_s.shape) != (M, kblocks(K)) or tuple(b_s.shape) != (kblocks(N), kblocks(K)):
        raise Dsfp8Error("scale shapes must be a_s [M, ceil(K/128)] and b_s [ceil(N/128), ceil(K/128)]")
    lib = _lib.load()
    c = _out(out, (M, N), torch.bfloat16, a.device, "out")
    wsb = lib.dsfp8_gemm_workspace_bytes(M, N, K)
    # zero-filled, as the split products' arrival counters require
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device=a.device) if wsb else None
    st = lib.dsfp8_gemm(a.data_ptr(), _ld(a), a_s.data_ptr(), ars, aks, b.data_ptr(), _ld(b), b_s.data_ptr(),
                        _ld(b_s), c.data_ptr(), _ld(c), M, N, K, _fmt(scale_fmt),
                        ws.data_ptr() if ws is not None else None, wsb, _stream(a))
    _check("gemm", st)
    return c


def grouped_gemm(a, a_s, b, b_s, offsets, out=None, workspace=None, scale_fmt="fp32"):
    """Per-expert product over row ranges: rows ``offsets[e]:offsets[e+1]`` of A use W[e].

    ``b`` is e4m3 ``[E, N, K]``, ``b_s`` fp32 ``[E, ceil(N/128), ceil(K/128)]``,
    ``offsets`` int32 ``[E+1]`` on the device.  Returns bf16 ``[M_total, N]``.
    ``scale_fmt`` as for :func:`gemm`.
    """
    a = _mat(_bytes(a), "a", (torch.uint8,))
    b = _mat(_bytes(b), "b", (torch.uint8,), dim=3)
    ars, aks = _scale_matrix(a_s, "a_s")
    _mat(b_s, "b_s", (torch.float32,), dim=3)
    if not offsets.is_cuda or offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise Dsfp8Error("offsets must be a contiguous int32 CUDA tensor of length E+1")
    M, K = a.shape
    E, N, K2 = b.shape
    if K2 != K or offsets.numel() != E + 1:
        raise Dsfp8Error("shape mismatch between a, b and offsets")
    if not b.is_contiguous() or not b_s.is_contiguous():
        raise Dsfp8Error("b and b_s need contiguous storage")
    if tuple(b_s.shape) != (E, kblocks(N), kblocks(K)) or tuple(a_s.shape) != (M, kblocks(K)):
        raise Dsfp8Error("scale shapes must be a_s [M, ceil(K/128)] and b_s [E, ceil(N/128), ceil(K/128)]")
    lib = _lib.load()
    c = _out(out, (M, N), torch.bfloat16, a.device, "out")
    wsb = lib.dsfp8_grouped_gemm_workspace_bytes(E, M, N, K)
    if workspace is None or workspace.numel() < wsb:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=a.device)
    st = lib.dsfp8_grouped_gemm(a.data_ptr(), _ld(a), a_s.data_ptr(), ars, aks, b.data_ptr(), K, b_s.data_ptr(),
                                kblocks(K), offsets.data_ptr(), E, M, N, K, c.data_ptr(), _ld(c), _fmt(scale_fmt),
                                workspace.data_ptr(), workspace.numel(), _stream(a))
    _check("grouped_gemm", st)
    return c


def _glu_outputs(M, F, device, out, return_h):
    yo, so = out if out is not None else (None, None)
    y = _out(yo, (M, F), torch.uint8, device, "y")
    s = _scales_out(so, M, kblocks(F), device)
    h = torch.empty((M, F), dtype=torch.bfloat16, device=device) if return_h else None
    return y, s, h


def gemm_silu_mul_act_quant(a, a_s, w13, w13_s, scale_fmt="fp32", return_h=False, out=None):
    """The gated up-projection in one kernel: ``act_quant(bf16(SiLU(h1) * h3))``
    with ``h1 = gemm(a, a_s, w1, s1)`` and ``h3 = gemm(a, a_s, w3, s3)``, where
    ``w13`` e4m3 ``[2F, K]`` stacks w1 over w3 and ``w13_s`` their scale grids
    ``[2F/128, ceil(K/128)]``.  Equal to :func:`gemm` followed by
    :func:`silu_mul_act_quant` on the two halves.  Returns ``(y, s)`` or
    ``(y, s, h)``; ``out`` may supply ``(y, s)``.  ``scale_fmt`` applies to the
    operand scales and to the scales produced."""
    a = _mat(_bytes(a), "a", (torch.uint8,))
    w = _mat(_bytes(w13), "w13", (torch.uint8,))
    ars, aks = _scale_matrix(a_s, "a_s")
    _mat(w13_s, "w13_s", (torch.float32,))
    M, K = a.shape
    N2, K2 = w.shape
    if K2 != K or N2 % 2:
        raise Dsfp8Error(f"w13 must be [2F, {K}], got {tuple(w.shape)}")
    F = N2 // 2
    if tuple(a_s.shape) != (M, kblocks(K)) or tuple(w13_s.shape) != (kblocks(N2), kblocks(K)):
        raise Dsfp8Error("scale shapes must be a_s [M, ceil(K/128)] and w13_s [2F/128, ceil(K/128)]")
    y, s, h = _glu_outputs(M, F, a.device, out, return_h)
    srs, sks = _scale_strides(s)
    st = _lib.load().dsfp8_gemm_silu_mul_act_quant(
        a.data_ptr(), _ld(a), a_s.data_ptr(), ars, aks, w.data_ptr(), _ld(w), w13_s.data_ptr(), _ld(w13_s),
        M, F, K, y.data_ptr(), _ld(y), s.data_ptr(), srs, sks, h.data_ptr() if h is not None else None, F,
        _fmt(scale_fmt), _stream(a))
    _check("gemm_silu_mul_act_quant", st)
    return (y, s, h) if return_h else (y, s)


def grouped_gemm_silu_mul_act_quant(a, a_s, w13, w13_s, offsets, scale_fmt="fp32", return_h=False, out=None,
                                    workspace=None, rows=None):
    """Grouped form of :func:`gemm_silu_mul_act_quant`: rows
    ``offsets[e]:offsets[e+1]`` of A use expert e's stacked ``w13[e]`` e4m3
    ``[2F, K]`` and ``w13_s[e]`` ``[2F/128, ceil(K/128)]``.

    ``rows`` (int32 CUDA tensor [M_total], optional): product row r reads row
    ``rows[r]`` of ``a`` and ``a_s`` (clamped to ``[0, a.shape[0])``), so the
    per-token quantised input feeds the experts without a gathered copy."""
    a = _mat(_bytes(a), "a", (torch.uint8,))
    w = _mat(_bytes(w13), "w13", (torch.uint8,), dim=3)
    ars, aks = _scale_matrix(a_s, "a_s")
    _mat(w13_s, "w13_s", (torch.float32,), dim=3)
    if not offsets.is_cuda or offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise Dsfp8Error("offsets must be a contiguous int32 CUDA tensor of length E+1")
    A_rows, K = a.shape
    if rows is not None:
        if not rows.is_cuda or rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
            raise Dsfp8Error("rows must be a contiguous 1-D int32 CUDA tensor")
        M = rows.numel()
    else:
        M = A_rows
    E, N2, K2 = w.shape
    if K2 != K or N2 % 2 or offsets.numel() != E + 1:
        raise Dsfp8Error("shape mismatch between a, w13 and offsets")
    if not w.is_contiguous() or not w13_s.is_contiguous():
        raise Dsfp8Error("w13 and w13_s need contiguous storage")
    F = N2 // 2
    if tuple(w13_s.shape) != (E, kblocks(N2), kblocks(K)) or tuple(a_s.shape) != (A_rows, kblocks(K)):
        raise Dsfp8Error("scale shapes must be a_s [rows of a, ceil(K/128)] and w13_s [E, 2F/128, ceil(K/128)]")
    lib = _lib.load()
    y, s, h = _glu_outputs(M, F, a.device, out, return_h)
    srs, sks = _scale_strides(s)
    wsb = lib.dsfp8_grouped_gemm_workspace_bytes(E, M, N2, K)
    if workspace is None or workspace.numel() < wsb:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=a.device)
    tail = (w.data_ptr(), K, w13_s.data_ptr(), kblocks(K), offsets.data_ptr(), E, M, F, K, y.data_ptr(), _ld(y),
            s.data_ptr(), srs, sks, h.data_ptr() if h is not None else None, F, _fmt(scale_fmt),
            workspace.data_ptr(), workspace.numel(), _stream(a))
    if rows is None:
        st = lib.dsfp8_grouped_gemm_silu_mul_act_quant(a.data_ptr(), _ld(a), a_s.data_ptr(), ars, aks, *tail)
    else:
        st = lib.dsfp8_grouped_gemm_silu_mul_act_quant_gather(a.data_ptr(), A_rows, _ld(a), a_s.data_ptr(), ars,
                                                              aks, rows.data_ptr(), *tail)
    _check("grouped_gemm_silu_mul_act_quant", st)
    return (y, s, h) if return_h else (y, s)


# ---- routed experts ------------------------------------------------------------------

def act_quant_rows(x, rows, scale_fmt="fp32", out=None):
    """``act_quant(x[rows])`` without forming the gathered copy: e4m3 ``[len(rows), K]``
    and its scales.  ``rows`` is an int32 CUDA tensor; entries are clamped to
    ``[0, x.shape[0])``."""
    x = _mat(x, "x", (torch.bfloat16,))
    if not rows.is_cuda or rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
        raise Dsfp8Error("rows must be a contiguous int32 CUDA tensor")
    T, K = x.shape
    M = rows.numel()
    y, s = (None, None) if out is None else out
    y = _out(y, (M, K), torch.uint8, x.device, "y")
    s = _scales_out(s, M, kblocks(K), x.device)
    srs, sks = _scale_strides(s)
    st = _lib.load().dsfp8_act_quant_rows(x.data_ptr(), T, _ld(x), rows.data_ptr(), M, K, y.data_ptr(), _ld(y),
                                          s.data_ptr(), srs, sks, _fmt(scale_fmt), _stream(x))
    _check("act_quant_rows", st)
    return y, s


def _int32_mat(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32 or t.dim() != 2:
        raise Dsfp8Error(f"{name} must be a 2-D int32 CUDA tensor")
    if t.numel() > 0 and t.stride(-1) != 1:
        raise Dsfp8Error(f"{name}: the last dimension needs stride 1")
    return t


def moe_route(indices, experts):
    """Row order of the grouped product for the gate's ``indices [T, k]`` (int32).

    Returns ``(offsets int32 [E+1], row_token int32 [T*k], token_rows int32 [T, k])``:
    rows ``offsets[e]:offsets[e+1]`` are expert e's (token, slot) pairs in row-major
    order, ``row_token[r]`` is the token of row r and ``token_rows[t, j]`` the row
    of pair (t, j) (-1 when its index is outside ``[0, E)``).
    """
    indices = _int32_mat(indices, "indices")
    T, k = indices.shape
    lib = _lib.load()
    dev = indices.device
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    row_token = torch.empty(T * k, dtype=torch.int32, device=dev)
    token_rows = torch.empty((T, k), dtype=torch.int32, device=dev)
    wsb = lib.dsfp8_moe_route_workspace_bytes(T, k, experts)
    ws = torch.empty(max(wsb, 4), dtype=torch.uint8, device=dev)
    st = lib.dsfp8_moe_route(indices.data_ptr(), T, k, _ld(indices), experts, offsets.data_ptr(),
                             row_token.data_ptr(), token_rows.data_ptr(), ws.data_ptr(), ws.numel(), _stream(indices))
    _check("moe_route", st)
    return offsets, row_token, token_rows


def moe_combine(yr, indices, weights, token_rows, out=None):
    """bf16 ``[T, D]``: per token, the bf16 sum over its experts (in increasing
    index) of ``bf16(yr[token_rows[t, j]] * weights[t, j])``, as the pages' loop
    accumulates ``y[idx] += expert(x[idx]) * weights[idx, top]``."""
    yr = _mat(yr, "yr", (torch.bfloat16,))
    indices = _int32_mat(indices, "indices")
    weights = _mat(weights, "weights", (torch.bfloat16,))
    token_rows = _int32_mat(token_rows, "token_rows")
    T, k = indices.shape
    if tuple(weights.shape) != (T, k) or tuple(token_rows.shape) != (T, k) or not token_rows.is_contiguous():
        raise Dsfp8Error("weights and token_rows must be [T, k] (token_rows contiguous) like indices")
    R, D = yr.shape
    out = _out(out, (T, D), torch.bfloat16, yr.device, "out")
    st = _lib.load().dsfp8_moe_combine(yr.data_ptr(), R, _ld(yr), indices.data_ptr(), _ld(indices),
                                       weights.data_ptr(), _ld(weights), token_rows.data_ptr(), T, k, D,
                                       out.data_ptr(), _ld(out), _stream(yr))
    _check("moe_combine", st)
    return out


# ---- int8 linear layer -----------------------------------------------------------------


def _is_mat(t, dtype, dim=2):
    """What `_mat` asks for, as one expression for calls whose cost counts."""
    return (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.dim() == dim
            and (t.is_contiguous() or t.stride(dim - 1) == 1 or t.numel() == 0))


def _need(t, name, dtype, dim=2):
    if not _is_mat(t, dtype, dim):
        _mat(t, name, (dtype,), dim)


def _row(t, n):
    """`_ld` of a matrix whose last dimension is n."""
    return n if t.is_contiguous() else _ld(t)


def _expert_ld(t, name):
    """Row stride of stacked matrices [E, rows, columns], whose rows must be evenly spaced over the experts."""
    if t.is_contiguous() or t.numel() == 0:
        return t.shape[2]
    E, rows, _ = t.shape
    of_expert, of_row, _ = t.stride()
    if E == 1:
        return of_row
    if rows > 1 and of_expert != rows * of_row:
        raise Dsfp8Error(f"{name}: experts must follow each other row by row")
    return of_expert // rows


def _same_device(dev, **others):
    for name, o in others.items():
        if o.get_device() != dev:
            raise Dsfp8Error(f"{name} must be on device {dev}, got {o.device}")


def _vec_f32(t, n, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or t.shape != (n,):
        raise Dsfp8Error(f"{name} must be a float32 CUDA tensor of shape ({n},)")
    if n > 1 and t.stride(0) != 1:
        raise Dsfp8Error(f"{name} needs stride 1")


def _workspace(ws, need, t):
    """The address and size of the caller's workspace, or of a new one."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=t.device)
        return ws, ws.data_ptr(), need
    if (not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.dtype != torch.uint8 or not ws.is_contiguous()
            or ws.get_device() != t.get_device()):
        raise Dsfp8Error(f"workspace must be a contiguous uint8 tensor on {t.device}")
    return ws, ws.data_ptr(), ws.numel()


def _launch(name, fn, dev, *args):
    """Call an entry point on the device's current stream, with that device current."""
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        _check(name, st)


def row_quant_i8(x, out=None):
    """Quantise fp32 or bf16 ``x [M, K]`` to int8 with one scale per row.

    Returns ``(y int8 [M, K], s float32 [M])`` with x ~= y * s[:, None]: the
    activations of a token, or the weights of an output channel.  ``out`` may
    supply preallocated ``(y, s)`` (row strides of y are honoured)."""
    _mat(x, "x", (torch.float32, torch.bfloat16))
    M, K = x.shape
    yo, so = out if out is not None else (None, None)
    y = _out(yo, (M, K), torch.int8, x.device, "y")
    s = _out(so, (M,), torch.float32, x.device, "s")
    _launch("row_quant_i8", _lib.load().dsfp8_row_quant_i8, x.get_device(), x.data_ptr(),
            0 if x.dtype == torch.float32 else 1, M, K, _ld(x), y.data_ptr(), _ld(y), s.data_ptr())
    return y, s


def _gate_pair(g, u):
    _need(g, "g", torch.bfloat16)
    _need(u, "u", torch.bfloat16)
    if g.shape != u.shape:
        raise Dsfp8Error(f"g and u must have the same shape, got {tuple(g.shape)} and {tuple(u.shape)}")
    _same_device(g.get_device(), u=u)


def silu_mul_row_quant_i8(g, u, out=None):
    """``row_quant_i8(SiLU(g) * u)`` in one pass over bf16 ``g`` and ``u`` (the gate
    is evaluated in fp32 and not rounded before the quantisation)."""
    _gate_pair(g, u)
    M, I = g.shape
    yo, so = out if out is not None else (None, None)
    y = _out(yo, (M, I), torch.int8, g.device, "y")
    s = _out(so, (M,), torch.float32, g.device, "s")
    _launch("silu_mul_row_quant_i8", _lib.load().dsfp8_silu_mul_row_quant_i8, g.get_device(), g.data_ptr(), _ld(g),
            u.data_ptr(), _ld(u), M, I, y.data_ptr(), _ld(y), s.data_ptr())
    return y, s


def gemm_i8(a, a_s, b, b_s, out=None):
    """bf16 ``C [M, N] = (A W^T) * a_s[:, None] * b_s`` of int8 ``A [M, K]`` and
    ``W [N, K]``, summed exactly; ``a_s [M]`` and ``b_s [N]`` are float32."""
    _need(a, "a", torch.int8)
    _need(b, "b", torch.int8)
    M, K = a.shape
    N, K2 = b.shape
    if K2 != K:
        raise Dsfp8Error(f"a and b disagree on K: {K} vs {K2}")
    _vec_f32(a_s, M, "a_s")
    _vec_f32(b_s, N, "b_s")
    dev = a.get_device()
    _same_device(dev, a_s=a_s, b=b, b_s=b_s)
    c = _out(out, (M, N), torch.bfloat16, a.device, "out")
    _launch("gemm_i8", _lib.load().dsfp8_gemm_i8, dev, a.data_ptr(), _ld(a), a_s.data_ptr(), b.data_ptr(), _ld(b),
            b_s.data_ptr(), c.data_ptr(), _ld(c), M, N, K)
    return c


def _linear_i8(name, x, u, w, w_s, out, workspace):
    _need(w, "w", torch.int8)
    M, K = x.shape
    N, K2 = w.shape
    if K2 != K:
        raise Dsfp8Error(f"the input and w disagree on K: {K} vs {K2}")
    _vec_f32(w_s, N, "w_s")
    dev = x.get_device()
    if w.get_device() != dev or w_s.get_device() != dev:
        _same_device(dev, w=w, w_s=w_s)
    lib = _lib.load()
    c = x.new_empty((M, N)) if out is None else _out(out, (M, N), torch.bfloat16, x.device, "out")
    ws, wp, wn = _workspace(workspace, lib.dsfp8_linear_i8_workspace_bytes(M, N, K, 0 if u is None else 1), x)
    tail = (w.data_ptr(), _row(w, K), w_s.data_ptr(), c.data_ptr(), _row(c, N), M, N, K, wp, wn)
    if u is None:
        _launch(name, lib.dsfp8_linear_i8, dev, x.data_ptr(), _row(x, K), *tail)
    else:
        _launch(name, lib.dsfp8_silu_mul_linear_i8, dev, x.data_ptr(), _row(x, K), u.data_ptr(), _row(u, K), *tail)
    return c


def linear_i8(x, w, w_s, out=None, workspace=None):
    """bf16 ``[M, N]``: ``gemm_i8(*row_quant_i8(x), w, w_s)`` in one call, for bf16
    ``x [M, K]`` and an int8 weight ``w [N, K]`` with a float32 scale per output
    channel, ``w_s [N]`` (as ``row_quant_i8`` of the real weight gives them)."""
    _need(x, "x", torch.bfloat16)
    return _linear_i8("linear_i8", x, None, w, w_s, out, workspace)


def linear_i8_workspace_bytes(M, N, K, gated=False):
    """Bytes of ``workspace`` that :func:`linear_i8` (``gated``: :func:`silu_mul_linear_i8`) needs; 0 for few rows."""
    return _lib.load().dsfp8_linear_i8_workspace_bytes(M, N, K, 1 if gated else 0)


def silu_mul_linear_i8(g, u, w, w_s, out=None, workspace=None):
    """The gated form of :func:`linear_i8`, the down-projection of a feed-forward
    layer: ``gemm_i8(*silu_mul_row_quant_i8(g, u), w, w_s)`` in one call."""
    _gate_pair(g, u)
    return _linear_i8("silu_mul_linear_i8", g, u, w, w_s, out, workspace)


# ---- routed experts for a few tokens ------------------------------------------------------

MOE_FEW_MAX_TOKENS = 64


def moe_few_workspace_bytes(T, k, F):
    """Bytes of ``workspace`` that :func:`moe_few` needs for T tokens of k experts with F hidden columns."""
    return _lib.load().dsfp8_moe_few_workspace_bytes(T, k, F)


def moe_few(x, w13, w13_s, w2, w2_s, indices, weights, out=None, workspace=None):
    """A whole routed-expert layer for at most 64 tokens, in two kernels: bf16
    ``[T, D]``, per token the sum over its slots of ``weights[t, j] * W2[e] h`` with
    ``h = SiLU(W1[e] x) * (W3[e] x)`` and ``e = indices[t, j]``; slots whose expert
    is outside ``[0, E)`` contribute nothing.

    ``x`` bf16 ``[T, D]``; ``w13 [E, 2F, D]`` stacks w1 over w3, ``w2 [E, D, F]``:
    either e4m3 (uint8 or float8_e4m3fn) with 128x128 block scales ``w13_s
    [E, ceil(2F/128), ceil(D/128)]`` and ``w2_s [E, ceil(D/128), ceil(F/128)]``, or
    int8 with channel scales ``w13_s [E, 2F]`` and ``w2_s [E, D]``; ``indices``
    int32 and ``weights`` bf16 ``[T, k]``.  Activations are not quantised.  The
    same call gives the same bytes; another routing of the other tokens may
    change the order of a token's fp32 sums."""
    _need(x, "x", torch.bfloat16)
    _mat(w13, "w13", (torch.uint8, torch.int8, torch.float8_e4m3fn), dim=3)
    i8 = w13.dtype == torch.int8
    if not _is_mat(w2, w13.dtype, 3):
        _mat(w2, "w2", (torch.int8,) if i8 else (torch.uint8, torch.float8_e4m3fn), dim=3)
    if not _is_mat(indices, torch.int32):
        _int32_mat(indices, "indices")
    _need(weights, "weights", torch.bfloat16)
    T, D = x.shape
    E, F2, D2 = w13.shape
    F = F2 // 2
    if D2 != D or F2 % 2 or w2.shape != (E, D, F):
        raise Dsfp8Error(f"w13 must be [E, 2F, {D}] and w2 [E, {D}, F], got {tuple(w13.shape)} and {tuple(w2.shape)}")
    k = indices.shape[1]
    if indices.shape[0] != T or weights.shape != (T, k):
        raise Dsfp8Error(f"indices and weights must be [{T}, k]")
    _need(w13_s, "w13_s", torch.float32, 2 if i8 else 3)
    _need(w2_s, "w2_s", torch.float32, 2 if i8 else 3)
    want13 = (E, F2) if i8 else (E, kblocks(F2), kblocks(D))
    want2 = (E, D) if i8 else (E, kblocks(D), kblocks(F))
    if w13_s.shape != want13 or w2_s.shape != want2:
        raise Dsfp8Error(f"scales must be w13_s {want13} and w2_s {want2}, got {tuple(w13_s.shape)} and "
                         f"{tuple(w2_s.shape)}")
    ld13, ld2 = _expert_ld(w13, "w13"), _expert_ld(w2, "w2")
    lds13 = _row(w13_s, F2) if i8 else _expert_ld(w13_s, "w13_s")
    lds2 = _row(w2_s, D) if i8 else _expert_ld(w2_s, "w2_s")
    dev = x.get_device()
    if not (w13.get_device() == w2.get_device() == w13_s.get_device() == w2_s.get_device() == indices.get_device()
            == weights.get_device() == dev):
        _same_device(dev, w13=w13, w13_s=w13_s, w2=w2, w2_s=w2_s, indices=indices, weights=weights)
    lib = _lib.load()
    out = x.new_empty((T, D)) if out is None else _out(out, (T, D), torch.bfloat16, x.device, "out")
    ws, wp, wn = _workspace(workspace, lib.dsfp8_moe_few_workspace_bytes(T, k, F), x)
    _launch("moe_few", lib.dsfp8_moe_few, dev, x.data_ptr(), _row(x, D), w13.data_ptr(), ld13, w13_s.data_ptr(), lds13,
            w2.data_ptr(), ld2, w2_s.data_ptr(), lds2, 1 if i8 else 0, indices.data_ptr(), _row(indices, k),
            weights.data_ptr(), _row(weights, k), T, k, E, D, F, out.data_ptr(), _row(out, D), wp, wn)
    return out
