"""The linear layer in 8-bit integers with a scale for each token and channel (binding of include/fp8bq_int8.h).

Codes are int8 [R, K], scales float32 [R]; a value is q[r, k] * s[r].  Raw entry points, tensors in place of pointers:

    fp8bq_quantize_int8(x, q, s)
    fp8bq_quantize_int8_t(x, qt, st, ws)
    fp8bq_gemm_int8(qa, sa, qb, sb, c, ws=None, accumulate=False)
    fp8bq_linear_int8(x, qw, sw, y, ws=None)
    fp8bq_grouped_gemm_int8(qa, sa, offsets, qw, sw, y, ws=None)
    fp8bq_grouped_linear_int8(x, offsets, qw, sw, y, ws=None)
    fp8bq_quantize_int8_t_workspace_size(R, C), fp8bq_{gemm,linear}_int8_workspace_size(M, N, K),
    fp8bq_grouped_{gemm,linear}_int8_workspace_size(E, T, N, K)

Allocating helpers:

    quantize_int8(x) -> (q [R, C], s [R])                      a scale for each row
    quantize_int8_t(x) -> (qt [C, 16 ceil(R/16)], st [C])      a scale for each column, codes transposed
    gemm_int8(qa, sa, qb, sb, out_dtype=bf16, out=None, ws=None, accumulate=False) -> [M, N]
    linear_int8(x, qw, sw, out_dtype=bf16, out=None, ws=None) -> y [M, N], x quantized in the call
    grouped_gemm_int8(qa, sa, offsets, qw, sw, out_dtype=bf16, out=None, ws=None) -> y [T, N]
    grouped_linear_int8(x, offsets, qw, sw, out_dtype=bf16, out=None, ws=None) -> y [T, N]

Training: fprop is linear_int8 (or gemm_int8 on row codes); dX = gemm_int8(rows of dY, columns of W) and
dW = gemm_int8(columns of dY, columns of X), with the quantizers' gradient taken straight through.
"""

import torch

from . import IN_BF16, IN_F32, OUT_BF16, OUT_F32, OUT_F32_ACCUM, _RESTYPES, _SIGS, _c_i64, _c_int, _c_sz, _c_vp, _entry, lib
from ._marshal import F32, HI, I8, experts, experts_of, matrix, on_its_device, space, stacked, stream, vector
from .mx import _output, _space

_OUT_WS = [_c_vp, _c_int, _c_i64, _c_vp, _c_sz, _c_vp]
_CODES = [_c_vp, _c_i64, _c_vp]
_VALUES = [_c_vp, _c_int, _c_i64]
_INPUT = [_c_vp, _c_int, _c_i64, _c_i64, _c_i64]
_SIGS.update({
    "fp8bq_quantize_int8": _INPUT + _CODES + [_c_vp],
    "fp8bq_quantize_int8_t": _INPUT + _CODES + [_c_vp, _c_sz, _c_vp],
    "fp8bq_gemm_int8": [_c_i64] * 3 + _CODES + _CODES + _OUT_WS,
    "fp8bq_linear_int8": [_c_i64] * 3 + _VALUES + _CODES + _OUT_WS,
    "fp8bq_grouped_gemm_int8": [_c_i64] * 4 + [_c_vp] + _CODES + _CODES + _OUT_WS,
    "fp8bq_grouped_linear_int8": [_c_i64] * 4 + [_c_vp] + _VALUES + _CODES + _OUT_WS,
    "fp8bq_quantize_int8_t_workspace_size": [_c_i64] * 2,
    "fp8bq_gemm_int8_workspace_size": [_c_i64] * 3,
    "fp8bq_linear_int8_workspace_size": [_c_i64] * 3,
    "fp8bq_grouped_gemm_int8_workspace_size": [_c_i64] * 4,
    "fp8bq_grouped_linear_int8_workspace_size": [_c_i64] * 4,
})
for _name in _SIGS:
    if "_int8" in _name and _name.endswith("_workspace_size"):
        _RESTYPES[_name] = _c_sz


def fp8bq_quantize_int8_t_workspace_size(R, C):
    return lib().fp8bq_quantize_int8_t_workspace_size(R, C)


def fp8bq_gemm_int8_workspace_size(M, N, K):
    return lib().fp8bq_gemm_int8_workspace_size(M, N, K)


def fp8bq_linear_int8_workspace_size(M, N, K):
    return lib().fp8bq_linear_int8_workspace_size(M, N, K)


def fp8bq_grouped_gemm_int8_workspace_size(E, T, N, K):
    return lib().fp8bq_grouped_gemm_int8_workspace_size(E, T, N, K)


def fp8bq_grouped_linear_int8_workspace_size(E, T, N, K):
    return lib().fp8bq_grouped_linear_int8_workspace_size(E, T, N, K)


def _in(t):
    return IN_BF16 if t.dtype == torch.bfloat16 else IN_F32


def _out(t, accumulate=False):
    return OUT_F32_ACCUM if accumulate else OUT_BF16 if t.dtype == torch.bfloat16 else OUT_F32


def _padded(R):
    return (R + 15) // 16 * 16


@on_its_device
@_entry
def fp8bq_quantize_int8(x, q, s):
    R, C = x.shape
    dev = x.get_device()
    xp, ldx = matrix(x, "x", (R, C), HI, dev)
    qp, ldq = matrix(q, "q", (R, C), I8, dev)
    return xp, _in(x), R, C, ldx, qp, ldq, vector(s, "s", R, F32, dev), stream(dev)


@on_its_device
@_entry
def fp8bq_quantize_int8_t(x, qt, st, ws):
    R, C = x.shape
    dev = x.get_device()
    xp, ldx = matrix(x, "x", (R, C), HI, dev)
    qtp, ldqt = matrix(qt, "qt", (C, _padded(R)), I8, dev)
    stp = vector(st, "st", C, F32, dev)
    wsp, wsb = space(ws, dev)
    return xp, _in(x), R, C, ldx, qtp, ldqt, stp, wsp, wsb, stream(dev)


@on_its_device
@_entry
def fp8bq_gemm_int8(qa, sa, qb, sb, c, ws=None, accumulate=False):
    M, K = qa.shape
    N = qb.shape[0]
    dev = qa.get_device()
    qap, ldqa = matrix(qa, "qa", (M, K), I8, dev)
    sap = vector(sa, "sa", M, F32, dev)
    qbp, ldqb = matrix(qb, "qb", (N, K), I8, dev)
    sbp = vector(sb, "sb", N, F32, dev)
    cp, ldc = matrix(c, "c", (M, N), F32 if accumulate else HI, dev)
    wsp, wsb = space(ws, dev)
    return M, N, K, qap, ldqa, sap, qbp, ldqb, sbp, cp, _out(c, accumulate), ldc, wsp, wsb, stream(dev)


@on_its_device
@_entry
def fp8bq_linear_int8(x, qw, sw, y, ws=None):
    M, K = x.shape
    N = qw.shape[0]
    dev = x.get_device()
    xp, ldx = matrix(x, "x", (M, K), HI, dev)
    qwp, ldqw = matrix(qw, "qw", (N, K), I8, dev)
    swp = vector(sw, "sw", N, F32, dev)
    yp, ldy = matrix(y, "y", (M, N), HI, dev)
    wsp, wsb = space(ws, dev)
    return M, N, K, xp, _in(x), ldx, qwp, ldqw, swp, yp, _out(y), ldy, wsp, wsb, stream(dev)


@on_its_device
@_entry
def fp8bq_grouped_gemm_int8(qa, sa, offsets, qw, sw, y, ws=None):
    T, K = qa.shape
    dev = qa.get_device()
    op, E = experts(offsets, dev)
    N = stacked(qw.shape[0], E, "qw")
    qap, ldqa = matrix(qa, "qa", (T, K), I8, dev)
    sap = vector(sa, "sa", T, F32, dev)
    qwp, ldqw = matrix(qw, "qw", (E * N, K), I8, dev)
    swp = vector(sw, "sw", E * N, F32, dev)
    yp, ldy = matrix(y, "y", (T, N), HI, dev)
    wsp, wsb = space(ws, dev)
    return E, T, N, K, op, qap, ldqa, sap, qwp, ldqw, swp, yp, _out(y), ldy, wsp, wsb, stream(dev)


@on_its_device
@_entry
def fp8bq_grouped_linear_int8(x, offsets, qw, sw, y, ws=None):
    T, K = x.shape
    dev = x.get_device()
    op, E = experts(offsets, dev)
    N = stacked(qw.shape[0], E, "qw")
    xp, ldx = matrix(x, "x", (T, K), HI, dev)
    qwp, ldqw = matrix(qw, "qw", (E * N, K), I8, dev)
    swp = vector(sw, "sw", E * N, F32, dev)
    yp, ldy = matrix(y, "y", (T, N), HI, dev)
    wsp, wsb = space(ws, dev)
    return E, T, N, K, op, xp, _in(x), ldx, qwp, ldqw, swp, yp, _out(y), ldy, wsp, wsb, stream(dev)


def _scales(x, n, elements):
    """n scales to be written; the calls write none over no elements, where the rule's is the smallest one."""
    return x.new_empty(n, dtype=torch.float32) if elements else x.new_full((n,), 1e-12, dtype=torch.float32)


def quantize_int8(x):
    R, C = x.shape
    q, s = x.new_empty((R, C), dtype=torch.int8), _scales(x, R, C)
    fp8bq_quantize_int8(x, q, s)
    return q, s


@on_its_device
def quantize_int8_t(x):
    R, C = x.shape
    qt, st = x.new_empty((C, _padded(R)), dtype=torch.int8), _scales(x, C, R)
    fp8bq_quantize_int8_t.__wrapped__(x, qt, st, _space("fp8bq_quantize_int8_t_workspace_size", x, R, C))
    return qt, st


@on_its_device
def gemm_int8(qa, sa, qb, sb, out_dtype=torch.bfloat16, out=None, ws=None, accumulate=False):
    """accumulate=True adds the result to `out` (FP32) instead of overwriting it."""
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate=True needs an FP32 `out` tensor holding the running sum")
    M, K = qa.shape
    N = qb.shape[0]
    c = _output(out, M, N, out_dtype, qa)
    if ws is None:
        ws = _space("fp8bq_gemm_int8_workspace_size", qa, M, N, K)
    fp8bq_gemm_int8.__wrapped__(qa, sa, qb, sb, c, ws, accumulate=accumulate)
    return c


@on_its_device
def linear_int8(x, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    M, K = x.shape
    N = qw.shape[0]
    y = _output(out, M, N, out_dtype, x)
    if ws is None:
        ws = _space("fp8bq_linear_int8_workspace_size", x, M, N, K)
    fp8bq_linear_int8.__wrapped__(x, qw, sw, y, ws)
    return y


@on_its_device
def grouped_gemm_int8(qa, sa, offsets, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    T, K = qa.shape
    E = experts_of(offsets)
    N = stacked(qw.shape[0], E, "qw")
    y = _output(out, T, N, out_dtype, qa)
    if ws is None:
        ws = _space("fp8bq_grouped_gemm_int8_workspace_size", qa, E, T, N, K)
    fp8bq_grouped_gemm_int8.__wrapped__(qa, sa, offsets, qw, sw, y, ws)
    return y


@on_its_device
def grouped_linear_int8(x, offsets, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    T, K = x.shape
    E = experts_of(offsets)
    N = stacked(qw.shape[0], E, "qw")
    y = _output(out, T, N, out_dtype, x)
    if ws is None:
        ws = _space("fp8bq_grouped_linear_int8_workspace_size", x, E, T, N, K)
    fp8bq_grouped_linear_int8.__wrapped__(x, offsets, qw, sw, y, ws)
    return y
