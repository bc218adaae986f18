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


# ---- MXFP4 ---------------------------------------------------------------------------------

MX_BLOCK = 32
_MX_VIEWS = tuple(getattr(torch, n) for n in ("float4_e2m1fn_x2", "float8_e8m0fnu") if hasattr(torch, n))


def mxblocks(n):
    return (int(n) + MX_BLOCK - 1) // MX_BLOCK


def mxfp4_empty(M, K, device, lead=()):
    """Storage for MXFP4 rows: codes uint8 ``[*lead, M, 16 * ceil(K/32)]`` and scale bytes uint8
    ``[*lead, M, ceil(K/32)]`` whose rows are a multiple of 16 bytes apart, as the products read them."""
    kb = mxblocks(K)
    q = torch.empty((*lead, M, 16 * kb), dtype=torch.uint8, device=device)
    s = torch.empty((*lead, M, (kb + 15) // 16 * 16), dtype=torch.uint8, device=device)
    return q, (s if kb % 16 == 0 else s[..., :kb])


def _mx(q, s, what):
    """Checked codes and scales of MXFP4 rows: ``(q, row stride, s, row stride)``."""
    if (isinstance(q, torch.Tensor) and isinstance(s, torch.Tensor) and q.dtype == torch.uint8 and s.dtype == torch.uint8
            and q.is_cuda and s.is_cuda and s.dim() == 2):
        rows, kb = s.shape      # the usual case, as one condition: what _mx_slow asks for
        if rows > 1 and kb > 0 and q.shape == (rows, 16 * kb):
            (ldq, qc), (lds, sc) = q.stride(), s.stride()
            if (qc == 1 and sc == 1 and not (ldq | lds) & 15 and lds >= kb
                    and (lds == kb or _mx_room(s, rows, lds, (kb + 15) & ~15))):
                return q, ldq, s, lds
    return _mx_slow(q, s, what, 2)


def _mx_room(s, rows, lds, pad):
    return s.untyped_storage().nbytes() >= s.storage_offset() + (rows - 1) * lds + pad


def _mx_slow(q, s, what, dim):
    if isinstance(q, torch.Tensor) and q.dtype in _MX_VIEWS:
        q = q.view(torch.uint8)
    if isinstance(s, torch.Tensor) and s.dtype in _MX_VIEWS:
        s = s.view(torch.uint8)
    _need(q, what, torch.uint8, dim)
    _need(s, what + "_s", torch.uint8, dim)
    kb = s.shape[-1]
    if q.shape[:-1] != s.shape[:-1] or q.shape[-1] != 16 * kb:
        raise Dsfp8Error(f"{what} and {what}_s must be [..., 16 * blocks] and [..., blocks], got {tuple(q.shape)} and "
                         f"{tuple(s.shape)}")
    ldq, pad = _mx_ld(q, what), (kb + 15) & ~15
    if s.numel() == 0:
        return q, ldq, s, pad
    rows = s.numel() // kb
    lds = pad if rows == 1 else _mx_ld(s, what + "_s")
    if lds % 16 or not _mx_room(s, rows, lds, pad):
        raise Dsfp8Error(f"{what}_s: rows of scales must be a multiple of 16 bytes apart, with room for {pad} bytes "
                         "each (mxfp4_empty allocates them so)")
    if ldq % 16:
        raise Dsfp8Error(f"{what}: rows of codes must be a multiple of 16 bytes apart")
    return q, ldq, s, lds


def _mx_ld(t, what):
    return _row(t, t.shape[-1]) if t.dim() == 2 else _expert_ld(t, what)


def _mx_out(out, M, K, t):
    """Codes and scales for M rows of K columns, each the caller's or new on t's device, with their row strides."""
    kb = (K + 31) >> 5
    q, s = (None, None) if out is None else out
    if s is None:
        pad = (kb + 15) & ~15
        s = t.new_empty((M, pad), dtype=torch.uint8)
        s = s if pad == kb else s.as_strided((M, kb), (pad, 1))
        if q is None:
            return t.new_empty((M, 16 * kb), dtype=torch.uint8), 16 * kb, s, pad
    if q is None:
        q = t.new_empty((M, 16 * kb), dtype=torch.uint8)
    _mat(q, "y", (torch.uint8,))
    _mat(s, "s", (torch.uint8,))
    if q.shape != (M, 16 * kb) or s.shape != (M, kb) or q.device != t.device or s.device != t.device:
        raise Dsfp8Error(f"out must be uint8 {(M, 16 * kb)} and {(M, kb)} on {t.device}, got {tuple(q.shape)} on "
                         f"{q.device} and {tuple(s.shape)} on {s.device}")
    return _mx(q, s, "y")


def mxfp4_quant(x, out=None):
    """Quantise fp32 or bf16 ``x [M, K]`` to MXFP4, in blocks of 32 columns.

    Returns ``(q uint8 [M, 16 * ceil(K/32)], s uint8 [M, ceil(K/32)])``: two e2m1
    codes a byte, the lower column in the low half (columns past K hold 0), and a
    scale byte per block, for x ~= code * 2^(s - 127).  ``out`` may supply ``(q,
    s)`` as :func:`mxfp4_empty` gives them (None for one that is to be new)."""
    if not _is_mat(x, torch.bfloat16):
        _mat(x, "x", (torch.float32, torch.bfloat16))
    M, K = x.shape
    q, ldq, s, lds = _mx_out(out, M, K, x)
    _launch("mxfp4_quant", _lib.load().dsfp8_mxfp4_quant, x.get_device(), x.data_ptr(),
            0 if x.dtype == torch.float32 else 1, M, K, _row(x, K), q.data_ptr(), ldq, s.data_ptr(), lds)
    return q, s


def silu_mul_mxfp4_quant(g, u, out=None):
    """``mxfp4_quant(SiLU(g) * u)`` in one pass over bf16 ``g`` and ``u`` (the gate is
    evaluated in fp32 and not rounded before the quantisation)."""
    _gate_pair(g, u)
    M, K = g.shape
    q, ldq, s, lds = _mx_out(out, M, K, g)
    _launch("silu_mul_mxfp4_quant", _lib.load().dsfp8_silu_mul_mxfp4_quant, g.get_device(), g.data_ptr(), _row(g, K),
            u.data_ptr(), _row(u, K), M, K, q.data_ptr(), ldq, s.data_ptr(), lds)
    return q, s


def mxfp4_dequant(q, s, K=None, out=None):
    """bf16 ``[M, K]``: the values of MXFP4 rows (K: their columns, by default all of their blocks')."""
    q, ldq, s, lds = _mx(q, s, "q")
    M, kb = s.shape
    K = MX_BLOCK * kb if K is None else int(K)
    if mxblocks(K) != kb:
        raise Dsfp8Error(f"{kb} blocks hold {MX_BLOCK * (kb - 1) + 1} to {MX_BLOCK * kb} columns, not {K}")
    dev = q.get_device()
    if s.get_device() != dev:
        _same_device(dev, s=s)
    out = q.new_empty((M, K), dtype=torch.bfloat16) if out is None else _out(out, (M, K), torch.bfloat16, q.device, "out")
    _launch("mxfp4_dequant", _lib.load().dsfp8_mxfp4_dequant, dev, q.data_ptr(), ldq, s.data_ptr(), lds, M, K,
            out.data_ptr(), _row(out, K))
    return out


def gemm_mxfp4(a, a_s, b, b_s, out=None):
    """bf16 ``C [M, N] = A W^T`` of MXFP4 rows ``(a, a_s)`` and an MXFP4 weight of N rows ``(b, b_s)``, both as
    :func:`mxfp4_quant` returns them."""
    a, lda, a_s, ldas = _mx(a, a_s, "a")
    b, ldb, b_s, ldbs = _mx(b, b_s, "b")
    M, kb = a_s.shape
    N = b_s.shape[0]
    if b_s.shape[1] != kb:
        raise Dsfp8Error(f"a and b disagree on K: {kb} vs {b_s.shape[1]} blocks")
    dev = a.get_device()
    if not (a_s.get_device() == b.get_device() == b_s.get_device() == dev):
        _same_device(dev, a_s=a_s, b=b, b_s=b_s)
    c = a.new_empty((M, N), dtype=torch.bfloat16) if out is None else _out(out, (M, N), torch.bfloat16, a.device, "out")
    _launch("gemm_mxfp4", _lib.load().dsfp8_gemm_mxfp4, dev, a.data_ptr(), lda, a_s.data_ptr(), ldas, b.data_ptr(), ldb,
            b_s.data_ptr(), ldbs, c.data_ptr(), _row(c, N), M, N, MX_BLOCK * kb)
    return c


def linear_mxfp4_workspace_bytes(M, N, K):
    """Bytes of ``workspace`` that :func:`linear_mxfp4` needs; 0 for few rows."""
    return _lib.load().dsfp8_linear_mxfp4_workspace_bytes(M, N, K)


def linear_mxfp4(x, w, w_s, out=None, workspace=None):
    """bf16 ``[M, N]``: ``gemm_mxfp4(*mxfp4_quant(x), w, w_s)`` in one call, for bf16 ``x [M, K]`` and an MXFP4
    weight of N rows (as ``mxfp4_quant`` of the real weight gives it)."""
    _need(x, "x", torch.bfloat16)
    w, ldw, w_s, ldws = _mx(w, w_s, "w")
    M, K = x.shape
    N = w_s.shape[0]
    if w_s.shape[1] != mxblocks(K):
        raise Dsfp8Error(f"x has {K} columns, {mxblocks(K)} blocks, and w {w_s.shape[1]} blocks")
    dev = x.get_device()
    if w.get_device() != dev or w_s.get_device() != dev:
        _same_device(dev, w=w, w_s=w_s)
    lib = _lib.load()
    c = x.new_empty((M, N)) if out is None else _out(out, (M, N), torch.bfloat16, x.device, "out")
    ws, wp, wn = _workspace(workspace, lib.dsfp8_linear_mxfp4_workspace_bytes(M, N, K), x)
    _launch("linear_mxfp4", lib.dsfp8_linear_mxfp4, dev, x.data_ptr(), _row(x, K), w.data_ptr(), ldw, w_s.data_ptr(), ldws,
            c.data_ptr(), _row(c, N), M, N, K, wp, wn)
    return c


def _int32_vec(t, n, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise Dsfp8Error(f"{name} must be a contiguous 1-D int32 CUDA tensor")
    if n is not None and t.numel() != n:
        raise Dsfp8Error(f"{name} must have {n} elements, got {t.numel()}")


def grouped_gemm_mxfp4(a, a_s, b, b_s, offsets, rows=None, out=None):
    """:func:`gemm_mxfp4` over per-expert row ranges: product rows ``offsets[e]:offsets[e+1]`` use the weight
    ``(b[e], b_s[e])``, codes ``[E, N, 16 * blocks]`` and scales ``[E, N, blocks]``; ``offsets`` int32 ``[E+1]`` on
    the device.  With ``rows`` (int32 ``[M_total]``) product row r reads row ``rows[r]`` of ``a`` (clamped), so the
    tokens' quantised rows feed the experts without a gathered copy.  Returns bf16 ``[M_total, N]``; rows past
    ``offsets[E]`` are left as they were (unspecified in a new output)."""
    a, lda, a_s, ldas = _mx(a, a_s, "a")
    b, ldb, b_s, ldbs = _mx_slow(b, b_s, "b", 3)
    E, N, kb = b_s.shape
    if a_s.shape[1] != kb:
        raise Dsfp8Error(f"a and b disagree on K: {a_s.shape[1]} vs {kb} blocks")
    _int32_vec(offsets, E + 1, "offsets")
    M = a.shape[0]
    dev = a.get_device()
    _same_device(dev, a_s=a_s, b=b, b_s=b_s, offsets=offsets)
    if rows is not None:
        _int32_vec(rows, None, "rows")
        _same_device(dev, rows=rows)
        M = rows.numel()
    c = a.new_empty((M, N), dtype=torch.bfloat16) if out is None else _out(out, (M, N), torch.bfloat16, a.device, "out")
    _launch("grouped_gemm_mxfp4", _lib.load().dsfp8_grouped_gemm_mxfp4, dev, a.data_ptr(), a.shape[0], lda,
            a_s.data_ptr(), ldas, rows.data_ptr() if rows is not None else None, b.data_ptr(), ldb, b_s.data_ptr(), ldbs,
            offsets.data_ptr(), E, M, N, MX_BLOCK * kb, c.data_ptr(), _row(c, N))
    return c


# ---- the choice of experts -------------------------------------------------------------------

_SCORES = {"sigmoid": 0, "softmax": 1}


def moe_gate(logits, k, bias=None, score="sigmoid", groups=1, top_groups=None, renormalize=True, scale=1.0, out=None):
    """The experts of each token: ``(indices int32 [T, k], weights bf16 [T, k])``, as the routed-expert calls take
    them, from the router's ``logits`` (fp32 or bf16 ``[T, E]``).

    ``score`` is "sigmoid" or "softmax"; ``bias`` (fp32 ``[E]``) is added for the choice alone.  With ``groups`` > 1
    only the experts of the ``top_groups`` best of ``groups`` equal groups are considered (a group's score: its best
    expert's, with a bias the sum of its two best).  Experts come in decreasing order, the lowest index first among
    equals.  ``weights`` are the chosen experts' scores times ``scale``, divided by their sum if ``renormalize``.
    An expert with a logit of -inf is never chosen; slots without an expert hold index -1 and weight 0."""
    if not _is_mat(logits, torch.float32):
        _mat(logits, "logits", (torch.float32, torch.bfloat16))
    if score not in _SCORES:
        raise Dsfp8Error(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if not hasattr(k, "__index__") or k < 1:
        raise Dsfp8Error(f"k must be a number of experts from 1 on, got {k!r}")
    T, E = logits.shape
    dev = logits.get_device()
    if bias is not None:
        _vec_f32(bias, E, "bias")
        if bias.get_device() != dev:
            _same_device(dev, bias=bias)
    if out is None:
        indices, weights = logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k), dtype=torch.bfloat16)
    else:
        indices = _out(out[0], (T, k), torch.int32, logits.device, "indices")
        weights = _out(out[1], (T, k), torch.bfloat16, logits.device, "weights")
    _launch("moe_gate", _lib.load().dsfp8_moe_gate, dev, logits.data_ptr(), 0 if logits.dtype == torch.float32 else 1,
            _row(logits, E), bias.data_ptr() if bias is not None else None, T, E, k, groups,
            groups if top_groups is None else top_groups, _SCORES[score], 1 if renormalize else 0, scale,
            indices.data_ptr(), _row(indices, k), weights.data_ptr(), _row(weights, k))
    return indices, weights


# ---- norms around a residual connection --------------------------------------------------------

_NORM_FMT = {None: 0, "e4m3": 1, "e4m3_ue8m0": 2, "mxfp4": 3}


def _norm_weight(w, D, name, dtype):
    if (not isinstance(w, torch.Tensor) or not w.is_cuda or w.dtype != dtype or w.shape != (D,)
            or not (D <= 1 or w.is_contiguous())):
        raise Dsfp8Error(f"{name} must be a {dtype} CUDA tensor of shape ({D},) with stride 1")


def add_rms_norm(x, weight, residual=None, post_weight=None, gate=None, scale=1.0, eps=1e-6, quant=None, out=None):
    """``y = rmsnorm(h) * weight`` with ``h = residual + scale * gate * t`` and ``t = x`` or, with ``post_weight``,
    ``rmsnorm(x) * post_weight``: the norm after a block (optional), its residual connection, and the norm before the
    next block, in one pass.  Without ``residual``, ``h = x`` (and no post_weight, gate or scale).

    ``x``, ``residual`` bf16 ``[T, D]``; ``gate`` bf16 ``[T, D]`` or ``[D]``; the weights ``[D]``, both bf16 or both
    fp32.  ``quant``: None for a bf16 y, "e4m3" or "e4m3_ue8m0" for :func:`act_quant`'s codes and scales of y, "mxfp4"
    for :func:`mxfp4_quant`'s.  Returns ``y`` or ``(y, s)``, followed by the new residual stream h (bf16) if there is
    a ``residual``.  ``out`` may supply the same tuple (``(y,)`` for y alone; None for one that is to be new); its h may
    be ``residual`` itself."""
    _need(x, "x", torch.bfloat16)
    T, D = x.shape
    dev = x.get_device()
    if quant not in _NORM_FMT:
        raise Dsfp8Error(f"quant must be one of {list(_NORM_FMT)}, got {quant!r}")
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (torch.bfloat16, torch.float32):
        raise Dsfp8Error("weight must be a bfloat16 or float32 tensor")
    _norm_weight(weight, D, "weight", weight.dtype)
    if weight.get_device() != dev:
        _same_device(dev, weight=weight)
    rp = gp = pp = None
    ldr = ldg = 0
    if post_weight is not None:
        _norm_weight(post_weight, D, "post_weight", weight.dtype)
        if post_weight.get_device() != dev:
            _same_device(dev, post_weight=post_weight)
        pp = post_weight.data_ptr()
    if residual is not None:
        _need(residual, "residual", torch.bfloat16)
        if residual.shape != x.shape:
            raise Dsfp8Error(f"residual must be {tuple(x.shape)}, got {tuple(residual.shape)}")
        if residual.get_device() != dev:
            _same_device(dev, residual=residual)
        rp, ldr = residual.data_ptr(), _row(residual, D)
    if gate is not None:
        g = gate[None] if isinstance(gate, torch.Tensor) and gate.dim() == 1 else gate
        _need(g, "gate", torch.bfloat16)
        if g.shape != (1 if gate.dim() == 1 else T, D):
            raise Dsfp8Error(f"gate must be {(T, D)} or {(D,)}, got {tuple(gate.shape)}")
        _same_device(dev, gate=gate)
        gp = g.data_ptr()
        ldg = 0 if gate.dim() == 1 or (T > 1 and g.stride(0) == 0) else _row(g, D)
    want = (1 if quant is None else 2) + (residual is not None)
    o = (None,) * want if out is None else tuple(out)
    if len(o) != want:
        raise Dsfp8Error(f"out must hold {want} tensors, got {len(o)}")
    s, sp, srs, sks = None, None, 0, 0
    if quant is None:
        y = x.new_empty((T, D)) if o[0] is None else _out(o[0], (T, D), torch.bfloat16, x.device, "y")
        ldy = _row(y, D)
    elif quant == "mxfp4":
        y, ldy, s, srs = _mx_out(o[:2], T, D, x)
        sp, sks = s.data_ptr(), 1
    else:
        y = x.new_empty((T, D), dtype=torch.uint8) if o[0] is None else _out(o[0], (T, D), torch.uint8, x.device, "y")
        ldy = _row(y, D)
        if o[1] is None:        # K-block-major, as new_scales
            srs, sks = 1, max(T, 1)
            s = x.new_empty_strided((T, kblocks(D)), (1, sks), dtype=torch.float32)
        else:
            s = _scales_out(o[1], T, kblocks(D), x.device)
            srs, sks = _scale_strides(s)
        sp = s.data_ptr()
    hp, h, ldh = None, None, 0
    if residual is not None:
        h = x.new_empty((T, D)) if o[-1] is None else _out(o[-1], (T, D), torch.bfloat16, x.device, "h")
        hp, ldh = h.data_ptr(), _row(h, D)
    _launch("add_rms_norm", _lib.load().dsfp8_add_rms_norm, dev, x.data_ptr(), _row(x, D), rp, ldr, gp, ldg, pp,
            weight.data_ptr(), 0 if weight.dtype == torch.float32 else 1, scale, eps, T, D, hp, ldh, y.data_ptr(), ldy,
            _NORM_FMT[quant], sp, srs, sks)
    got = (y,) if s is None else (y, s)
    got = got if h is None else got + (h,)
    return got if len(got) > 1 else y
