"""The linear layer in microscaled 4-bit floating point (binding of include/fp8bq_mx.h).

Codes are uint8 [R, K / 2] (two values a byte), scales uint8 [ceil(K / 128), R, 4]: byte [k / 128, r, (k / 32) % 4]
is the E8M0 scale of row r's block k / 32.  Raw entry points, tensors in place of pointers:

    fp8bq_quantize_mxfp4(x, q, s, qt, st)        (q and s, or qt and st, may be None)
    fp8bq_gemm_mxfp4(qa, sa, qb, sb, c, ws=None, accumulate=False)
    fp8bq_linear_mxfp4(x, qw, sw, y, ws=None)
    fp8bq_grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, y, ws=None)
    fp8bq_grouped_linear_mxfp4(x, offsets, qw, sw, y, ws=None)
    fp8bq_{gemm,linear}_mxfp4_workspace_size(M, N, K), fp8bq_grouped_{gemm,linear}_mxfp4_workspace_size(E, T, N, K)

Allocating helpers:

    quantize_mxfp4(x) -> (q [R, C/2], s [ceil(C/128), R, 4])                 blocks along the rows
    quantize_mxfp4_t(x) -> (qt [C, 16 ceil(R/32)], st [ceil(R/128), C, 4])   blocks down the columns, transposed
    quantize_mxfp4_dual(x) -> (q, s, qt, st), one pass over x
    gemm_mxfp4(qa, sa, qb, sb, out_dtype=bf16, out=None, ws=None, accumulate=False) -> [M, N]
    linear_mxfp4(x, qw, sw, out_dtype=bf16, out=None, ws=None) -> y [M, N], x quantized in the call
    grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, out_dtype=bf16, out=None, ws=None) -> y [T, N]
    grouped_linear_mxfp4(x, offsets, qw, sw, out_dtype=bf16, out=None, ws=None) -> y [T, N]

Training: fprop is linear_mxfp4 (or gemm_mxfp4 on row codes); dX = gemm_mxfp4(rows of dY, columns of W) and
dW = gemm_mxfp4(columns of dY, columns of X), with the quantizers' gradient taken straight through.
"""

import functools

import torch

from . import OUT_BF16, OUT_F32, OUT_F32_ACCUM, IN_BF16, IN_F32, _RESTYPES, _SIGS, _c_i64, _c_int, _c_sz, _c_vp, _entry, lib
from ._marshal import F32, HI, NONE, U8, experts, experts_of, matrix, scale_words, space, stacked, stream

_OUT_WS = [_c_vp, _c_int, _c_i64, _c_vp, _c_sz, _c_vp]
_CODES = [_c_vp, _c_i64, _c_vp, _c_i64]
_VALUES = [_c_vp, _c_int, _c_i64]
_SIGS.update({
    "fp8bq_quantize_mxfp4": [_c_vp, _c_int, _c_i64, _c_i64, _c_i64] + _CODES + _CODES + [_c_vp],
    "fp8bq_gemm_mxfp4": [_c_i64] * 3 + _CODES + _CODES + _OUT_WS,
    "fp8bq_linear_mxfp4": [_c_i64] * 3 + _VALUES + _CODES + _OUT_WS,
    "fp8bq_grouped_gemm_mxfp4": [_c_i64] * 4 + [_c_vp] + _CODES + _CODES + _OUT_WS,
    "fp8bq_grouped_linear_mxfp4": [_c_i64] * 4 + [_c_vp] + _VALUES + _CODES + _OUT_WS,
    "fp8bq_gemm_mxfp4_workspace_size": [_c_i64] * 3,
    "fp8bq_linear_mxfp4_workspace_size": [_c_i64] * 3,
    "fp8bq_grouped_gemm_mxfp4_workspace_size": [_c_i64] * 4,
    "fp8bq_grouped_linear_mxfp4_workspace_size": [_c_i64] * 4,
})
for _name in _SIGS:
    if _name.endswith("_mxfp4_workspace_size"):
        _RESTYPES[_name] = _c_sz


def fp8bq_gemm_mxfp4_workspace_size(M, N, K):
    return lib().fp8bq_gemm_mxfp4_workspace_size(M, N, K)


def fp8bq_linear_mxfp4_workspace_size(M, N, K):
    return lib().fp8bq_linear_mxfp4_workspace_size(M, N, K)


def fp8bq_grouped_gemm_mxfp4_workspace_size(E, T, N, K):
    return lib().fp8bq_grouped_gemm_mxfp4_workspace_size(E, T, N, K)


def fp8bq_grouped_linear_mxfp4_workspace_size(E, T, N, K):
    return lib().fp8bq_grouped_linear_mxfp4_workspace_size(E, T, N, K)


def _words(n):
    return (n + 127) // 128


def _in(t):
    return IN_BF16 if t.dtype == torch.bfloat16 else IN_F32


def _out(t, accumulate=False):
    return OUT_F32_ACCUM if accumulate else OUT_BF16 if t.dtype == torch.bfloat16 else OUT_F32


@_entry
def fp8bq_quantize_mxfp4(x, q, s, qt, st):
    R, C = x.shape
    dev = x.get_device()
    xp, ldx = matrix(x, "x", (R, C), HI, dev)
    qp, ldq = matrix(q, "q", (R, C // 2), U8, dev) if q is not None else NONE
    sp, lds = scale_words(s, "s", (_words(C), R, 4), dev) if s is not None else NONE
    qtp, ldqt = matrix(qt, "qt", (C, (R + 31) // 32 * 16), U8, dev) if qt is not None else NONE
    stp, ldst = scale_words(st, "st", (_words(R), C, 4), dev) if st is not None else NONE
    return xp, _in(x), R, C, ldx, qp, ldq, sp, lds, qtp, ldqt, stp, ldst, stream(dev)


@_entry
def fp8bq_gemm_mxfp4(qa, sa, qb, sb, c, ws=None, accumulate=False):
    M, K2 = qa.shape
    N = qb.shape[0]
    dev = qa.get_device()
    W = _words(2 * K2)
    qap, ldqa = matrix(qa, "qa", (M, K2), U8, dev)
    sap, ldsa = scale_words(sa, "sa", (W, M, 4), dev)
    qbp, ldqb = matrix(qb, "qb", (N, K2), U8, dev)
    sbp, ldsb = scale_words(sb, "sb", (W, N, 4), dev)
    cp, ldc = matrix(c, "c", (M, N), F32 if accumulate else HI, dev)
    wsp, wsb = space(ws, dev)
    return M, N, 2 * K2, qap, ldqa, sap, ldsa, qbp, ldqb, sbp, ldsb, cp, _out(c, accumulate), ldc, wsp, wsb, stream(dev)


@_entry
def fp8bq_linear_mxfp4(x, qw, sw, y, ws=None):
    M, K = x.shape
    N = qw.shape[0]
    dev = x.get_device()
    xp, ldx = matrix(x, "x", (M, K), HI, dev)
    qwp, ldqw = matrix(qw, "qw", (N, K // 2), U8, dev)
    swp, ldsw = scale_words(sw, "sw", (_words(K), N, 4), dev)
    yp, ldy = matrix(y, "y", (M, N), HI, dev)
    wsp, wsb = space(ws, dev)
    return M, N, K, xp, _in(x), ldx, qwp, ldqw, swp, ldsw, yp, _out(y), ldy, wsp, wsb, stream(dev)


@_entry
def fp8bq_grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, y, ws=None):
    T, K2 = qa.shape
    dev = qa.get_device()
    op, E = experts(offsets, dev)
    N = stacked(qw.shape[0], E, "qw")
    W = _words(2 * K2)
    qap, ldqa = matrix(qa, "qa", (T, K2), U8, dev)
    sap, ldsa = scale_words(sa, "sa", (W, T, 4), dev)
    qwp, ldqw = matrix(qw, "qw", (E * N, K2), U8, dev)
    swp, ldsw = scale_words(sw, "sw", (W, E * N, 4), dev)
    yp, ldy = matrix(y, "y", (T, N), HI, dev)
    wsp, wsb = space(ws, dev)
    return E, T, N, 2 * K2, op, qap, ldqa, sap, ldsa, qwp, ldqw, swp, ldsw, yp, _out(y), ldy, wsp, wsb, stream(dev)


@_entry
def fp8bq_grouped_linear_mxfp4(x, offsets, qw, sw, y, ws=None):
    T, K = x.shape
    dev = x.get_device()
    op, E = experts(offsets, dev)
    N = stacked(qw.shape[0], E, "qw")
    xp, ldx = matrix(x, "x", (T, K), HI, dev)
    qwp, ldqw = matrix(qw, "qw", (E * N, K // 2), U8, dev)
    swp, ldsw = scale_words(sw, "sw", (_words(K), E * N, 4), dev)
    yp, ldy = matrix(y, "y", (T, N), HI, dev)
    wsp, wsb = space(ws, dev)
    return E, T, N, K, op, xp, _in(x), ldx, qwp, ldqw, swp, ldsw, yp, _out(y), ldy, wsp, wsb, stream(dev)


def _codes(R, K, like):
    return like.new_empty((R, K // 2), dtype=torch.uint8), like.new_empty((_words(K), R, 4), dtype=torch.uint8)


def quantize_mxfp4(x):
    q, s = _codes(*x.shape, x)
    fp8bq_quantize_mxfp4(x, q, s, None, None)
    return q, s


def quantize_mxfp4_t(x):
    R, C = x.shape
    qt, st = _codes(C, (R + 31) // 32 * 32, x)
    fp8bq_quantize_mxfp4(x, None, None, qt, st)
    return qt, st


def quantize_mxfp4_dual(x):
    R, C = x.shape
    q, s = _codes(R, C, x)
    qt, st = _codes(C, (R + 31) // 32 * 32, x)
    fp8bq_quantize_mxfp4(x, q, s, qt, st)
    return q, s, qt, st


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


@functools.lru_cache(maxsize=4096)
def _ws_bytes(op, device, *sizes):
    """Workspace of an operation at these sizes on the current device, of that index: a function of these alone."""
    return getattr(lib(), op)(*sizes)


def _space(op, like, *sizes):
    n = _ws_bytes(op, _current_device() if like.is_cuda else -1, *sizes)
    return like.new_empty(n, dtype=torch.uint8) if n else None


def _output(out, M, N, dtype, like):
    return out if out is not None else like.new_empty((M, N), dtype=dtype)


def gemm_mxfp4(qa, sa, qb, sb, out_dtype=torch.bfloat16, out=None, ws=None, accumulate=False):
    """accumulate=True adds the result to `out` (FP32) instead of overwriting it."""
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate=True needs an FP32 `out` tensor holding the running sum")
    M, K2 = qa.shape
    N = qb.shape[0]
    c = _output(out, M, N, out_dtype, qa)
    if ws is None:
        ws = _space("fp8bq_gemm_mxfp4_workspace_size", qa, M, N, 2 * K2)
    fp8bq_gemm_mxfp4(qa, sa, qb, sb, c, ws, accumulate=accumulate)
    return c


def linear_mxfp4(x, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    M, K = x.shape
    N = qw.shape[0]
    y = _output(out, M, N, out_dtype, x)
    if ws is None:
        ws = _space("fp8bq_linear_mxfp4_workspace_size", x, M, N, K)
    fp8bq_linear_mxfp4(x, qw, sw, y, ws)
    return y


def grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    T, K2 = qa.shape
    E = experts_of(offsets)
    N = stacked(qw.shape[0], E, "qw")
    y = _output(out, T, N, out_dtype, qa)
    if ws is None:
        ws = _space("fp8bq_grouped_gemm_mxfp4_workspace_size", qa, E, T, N, 2 * K2)
    fp8bq_grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, y, ws)
    return y


def grouped_linear_mxfp4(x, offsets, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    T, K = x.shape
    E = experts_of(offsets)
    N = stacked(qw.shape[0], E, "qw")
    y = _output(out, T, N, out_dtype, x)
    if ws is None:
        ws = _space("fp8bq_grouped_linear_mxfp4_workspace_size", x, E, T, N, K)
    fp8bq_grouped_linear_mxfp4(x, offsets, qw, sw, y, ws)
    return y
