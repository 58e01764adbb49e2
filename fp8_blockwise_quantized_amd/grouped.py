"""The FP8 blockwise linear layer grouped by expert (binding of include/fp8bq_grouped.h).

Tokens sorted by expert; offsets [E + 1] int64 on the device (expert e: rows offsets[e] .. offsets[e+1]-1);
the experts' weights stacked, W [E N, K].  Raw entry points, tensors in place of pointers:

    fp8bq_quantize_act_grouped(x, offsets, fmt_rows, q, s, fmt_cols, qt, st)     (q and s may be None)
    fp8bq_grouped_gemm_fprop(qx, sx, fx, offsets, qw, sw, fw, y)
    fp8bq_grouped_gemm_dgrad(qdy, sdy, fdy, offsets, qwt, sw, fw, dx)
    fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fdy, qxt, sxt, fx, offsets, dw, accumulate=False, ws=None)
    fp8bq_grouped_gemm_wgrad_workspace_size(E, padded, N, K)   (without ws no expert's contraction is split)
    fp8bq_grouped_padded_rows(T, E)

Allocating helpers:

    quantize_act_grouped_128x1(x, offsets, fmt=E4M3) -> (qt [C, padded] uint8, st [padded/128, C] float32)
    quantize_act_grouped_dual(x, offsets, fmt_rows=E4M3, fmt_cols=E4M3) -> (q, s, qt, st), one pass over x
    grouped_gemm_fprop(qx, sx, offsets, qw, sw, fx=E4M3, fw=E4M3, out_dtype=bf16, out=None) -> y [T, N]
    grouped_gemm_dgrad(qdy, sdy, offsets, qwt, sw, fdy=E4M3, fw=E4M3, out_dtype=bf16, out=None) -> dx [T, K]
    grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offsets, fdy=E4M3, fx=E4M3, out_dtype=bf16, out=None,
                       accumulate=False, ws=None) -> dw [E N, K]

Rows of y and dx that belong to no expert are left as they are (undefined in a tensor made here).
"""

import torch

from . import (E4M3, IN_BF16, IN_F32, OUT_BF16, OUT_F32, OUT_F32_ACCUM, _c_i64, _c_int, _c_sz, _c_vp, _entry, _pad4,
               _RESTYPES, _SIGS, lib)
from ._marshal import F32, HI, NONE, U8, experts, experts_of, matrix, space, stacked, stream

MAX_EXPERTS = 512

_GEMM = [_c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_i64,
         _c_int, _c_vp, _c_int, _c_i64, _c_vp]
_SIGS.update({
    "fp8bq_grouped_padded_rows": [_c_i64, _c_i64],
    "fp8bq_quantize_act_grouped": [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_vp,
                                   _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp],
    "fp8bq_grouped_gemm_fprop": _GEMM,
    "fp8bq_grouped_gemm_dgrad": _GEMM,
    "fp8bq_grouped_gemm_wgrad": _GEMM[:-1] + [_c_vp, _c_sz, _c_vp],
    "fp8bq_grouped_gemm_wgrad_workspace_size": [_c_i64] * 4,
})
_RESTYPES["fp8bq_grouped_padded_rows"] = _c_i64
_RESTYPES["fp8bq_grouped_gemm_wgrad_workspace_size"] = _c_sz


def fp8bq_grouped_padded_rows(T, E):
    return int(lib().fp8bq_grouped_padded_rows(int(T), int(E)))


def fp8bq_grouped_gemm_wgrad_workspace_size(E, padded, N, K):
    return lib().fp8bq_grouped_gemm_wgrad_workspace_size(E, padded, N, K)


def _out(t, accumulate=False):
    return OUT_F32_ACCUM if accumulate else OUT_BF16 if t.dtype == torch.bfloat16 else OUT_F32


@_entry
def fp8bq_quantize_act_grouped(x, offsets, fmt_rows, q, s, fmt_cols, qt, st):
    T, C = x.shape
    dev = x.get_device()
    op, E = experts(offsets, dev)
    if not isinstance(qt, torch.Tensor) or qt.dim() != 2:
        raise TypeError("qt must be a 2-D torch tensor")
    padded = qt.shape[1]
    xp, ldx = matrix(x, "x", (T, C), HI, dev)
    qp, ldq = matrix(q, "q", (T, C), U8, dev) if q is not None else NONE
    sp, lds = matrix(s, "s", (C // 128, T), F32, dev) if s is not None else NONE
    qtp, ldqt = matrix(qt, "qt", (C, padded), U8, dev)
    stp, ldst = matrix(st, "st", (padded // 128, C), F32, dev)
    return (xp, IN_BF16 if x.dtype == torch.bfloat16 else IN_F32, T, C, ldx, op, E, fmt_rows, qp, ldq, sp, lds, fmt_cols,
            qtp, ldqt, stp, ldst, padded, stream(dev))


@_entry
def fp8bq_grouped_gemm_fprop(qx, sx, fx, offsets, qw, sw, fw, y):
    T, K = qx.shape
    dev = qx.get_device()
    op, E = experts(offsets, dev)
    N = stacked(qw.shape[0], E, "qw")
    qxp, ldqx = matrix(qx, "qx", (T, K), U8, dev)
    sxp, ldsx = matrix(sx, "sx", (K // 128, T), F32, dev)
    qwp, ldqw = matrix(qw, "qw", (E * N, K), U8, dev)
    swp, ldsw = matrix(sw, "sw", (E * N // 128, K // 128), F32, dev)
    yp, ldy = matrix(y, "y", (T, N), HI, dev)
    return E, T, N, K, op, qxp, ldqx, sxp, ldsx, fx, qwp, ldqw, swp, ldsw, fw, yp, _out(y), ldy, stream(dev)


@_entry
def fp8bq_grouped_gemm_dgrad(qdy, sdy, fdy, offsets, qwt, sw, fw, dx):
    T, N = qdy.shape
    dev = qdy.get_device()
    op, E = experts(offsets, dev)
    K = qwt.shape[0]
    qdyp, ldqdy = matrix(qdy, "qdy", (T, N), U8, dev)
    sdyp, ldsdy = matrix(sdy, "sdy", (N // 128, T), F32, dev)
    qwtp, ldqwt = matrix(qwt, "qwt", (K, E * N), U8, dev)
    swp, ldsw = matrix(sw, "sw", (E * N // 128, K // 128), F32, dev)
    dxp, lddx = matrix(dx, "dx", (T, K), HI, dev)
    return E, T, N, K, op, qdyp, ldqdy, sdyp, ldsdy, fdy, qwtp, ldqwt, swp, ldsw, fw, dxp, _out(dx), lddx, stream(dev)


@_entry
def fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fdy, qxt, sxt, fx, offsets, dw, accumulate=False, ws=None):
    N, padded = qdyt.shape
    dev = qdyt.get_device()
    op, E = experts(offsets, dev)
    K = qxt.shape[0]
    qdytp, ldqdyt = matrix(qdyt, "qdyt", (N, padded), U8, dev)
    sdytp, ldsdyt = matrix(sdyt, "sdyt", (padded // 128, N), F32, dev)
    qxtp, ldqxt = matrix(qxt, "qxt", (K, padded), U8, dev)
    sxtp, ldsxt = matrix(sxt, "sxt", (padded // 128, K), F32, dev)
    dwp, lddw = matrix(dw, "dw", (E * N, K), F32 if accumulate else HI, dev)
    wsp, ws_bytes = space(ws, dev)
    return (E, padded, N, K, op, qdytp, ldqdyt, sdytp, ldsdyt, fdy, qxtp, ldqxt, sxtp, ldsxt, fx, dwp,
            _out(dw, accumulate), lddw, wsp, ws_bytes, stream(dev))


def _cols_outputs(x, offsets):
    T, C = x.shape
    padded = fp8bq_grouped_padded_rows(T, experts_of(offsets))
    return x.new_empty((C, padded), dtype=torch.uint8), x.new_empty((padded // 128, C), dtype=torch.float32)


def quantize_act_grouped_128x1(x, offsets, fmt=E4M3):
    qt, st = _cols_outputs(x, offsets)
    fp8bq_quantize_act_grouped(x, offsets, E4M3, None, None, fmt, qt, st)
    return qt, st


def quantize_act_grouped_dual(x, offsets, fmt_rows=E4M3, fmt_cols=E4M3):
    """(q, s) of quantize_act_1x128(x, fmt_rows) and (qt, st) of quantize_act_grouped_128x1(x, offsets,
    fmt_cols) from one pass over x."""
    T, C = x.shape
    q = x.new_empty((T, C), dtype=torch.uint8)
    s = x.new_empty((C // 128, _pad4(T)), dtype=torch.float32)
    if s.shape[1] != T:
        s = s[:, :T]
    qt, st = _cols_outputs(x, offsets)
    fp8bq_quantize_act_grouped(x, offsets, fmt_rows, q, s, fmt_cols, qt, st)
    return q, s, qt, st


def grouped_gemm_fprop(qx, sx, offsets, qw, sw, fx=E4M3, fw=E4M3, out_dtype=torch.bfloat16, out=None):
    N = stacked(qw.shape[0], experts_of(offsets), "qw")
    y = out if out is not None else qx.new_empty((qx.shape[0], N), dtype=out_dtype)
    fp8bq_grouped_gemm_fprop(qx, sx, fx, offsets, qw, sw, fw, y)
    return y


def grouped_gemm_dgrad(qdy, sdy, offsets, qwt, sw, fdy=E4M3, fw=E4M3, out_dtype=torch.bfloat16, out=None):
    dx = out if out is not None else qdy.new_empty((qdy.shape[0], qwt.shape[0]), dtype=out_dtype)
    fp8bq_grouped_gemm_dgrad(qdy, sdy, fdy, offsets, qwt, sw, fw, dx)
    return dx


def grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offsets, fdy=E4M3, fx=E4M3, out_dtype=torch.bfloat16, out=None,
                       accumulate=False, ws=None):
    """accumulate=True adds the result to `out` (an FP32 main-grad buffer) instead of overwriting it.  ws: a uint8
    tensor of the workspace size (made here if None)."""
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate=True needs an FP32 `out` tensor holding the running sum")
    E = experts_of(offsets)
    N, padded = qdyt.shape
    K = qxt.shape[0]
    dw = out if out is not None else qdyt.new_empty((E * N, K), dtype=out_dtype)
    if ws is None:
        size = fp8bq_grouped_gemm_wgrad_workspace_size(E, padded, N, K)
        ws = qdyt.new_empty(size) if size else None
    fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fdy, qxt, sxt, fx, offsets, dw, accumulate=accumulate, ws=ws)
    return dw
