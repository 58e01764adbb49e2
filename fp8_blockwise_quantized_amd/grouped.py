"""The FP8 blockwise linear layer grouped by expert (binding of include/fp8bq_grouped.h).

Tokens sorted by expert; offsets [E + 1] int64 on the device (expert e: rows offsets[e] .. offsets[e+1]-1);
the experts' weights stacked, W [E N, K].  Raw entry points, tensors in place of pointers:

    fp8bq_quantize_act_grouped(x, offsets, fmt_rows, q, s, fmt_cols, qt, st)     (q and s may be None)
    fp8bq_grouped_gemm_fprop(qx, sx, fx, offsets, qw, sw, fw, y)
    fp8bq_grouped_gemm_dgrad(qdy, sdy, fdy, offsets, qwt, sw, fw, dx)
    fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fdy, qxt, sxt, fx, offsets, dw, accumulate=False)
    fp8bq_grouped_padded_rows(T, E)

Allocating helpers:

    quantize_act_grouped_128x1(x, offsets, fmt=E4M3) -> (qt [C, padded] uint8, st [padded/128, C] float32)
    quantize_act_grouped_dual(x, offsets, fmt_rows=E4M3, fmt_cols=E4M3) -> (q, s, qt, st), one pass over x
    grouped_gemm_fprop(qx, sx, offsets, qw, sw, fx=E4M3, fw=E4M3, out_dtype=bf16, out=None) -> y [T, N]
    grouped_gemm_dgrad(qdy, sdy, offsets, qwt, sw, fdy=E4M3, fw=E4M3, out_dtype=bf16, out=None) -> dx [T, K]
    grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offsets, fdy=E4M3, fx=E4M3, out_dtype=bf16, out=None,
                       accumulate=False) -> dw [E N, K]

Rows of y and dx that belong to no expert are left as they are (undefined in a tensor made here).
"""

import torch

from . import (_F32, _HI, _U8, E4M3, OUT_F32_ACCUM, _c_i64, _c_int, _c_vp, _entry, _expect_all, _in_type, _ld,
               _out_type, _pad4, _ptr, _RESTYPES, _SIGS, _stream, lib)

MAX_EXPERTS = 512

_GEMM = [_c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_i64,
         _c_int, _c_vp, _c_int, _c_i64, _c_vp]
_SIGS.update({
    "fp8bq_grouped_padded_rows": [_c_i64, _c_i64],
    "fp8bq_quantize_act_grouped": [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_vp,
                                   _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp],
    "fp8bq_grouped_gemm_fprop": _GEMM,
    "fp8bq_grouped_gemm_dgrad": _GEMM,
    "fp8bq_grouped_gemm_wgrad": _GEMM,
})
_RESTYPES["fp8bq_grouped_padded_rows"] = _c_i64

_I64 = (torch.int64,)


def fp8bq_grouped_padded_rows(T, E):
    return int(lib().fp8bq_grouped_padded_rows(int(T), int(E)))


def _experts(offsets):
    """The number of experts E of an offsets tensor of E + 1 entries."""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be a 1-D tensor of E + 1 entries")
    if not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous")
    return offsets.numel() - 1


def _stacked(rows, E, what):
    if rows % E:
        raise ValueError(f"{what}: {rows} stacked rows do not split over {E} experts")
    return rows // E


@_entry
def fp8bq_quantize_act_grouped(x, offsets, fmt_rows, q, s, fmt_cols, qt, st):
    T, C = x.shape
    E = _experts(offsets)
    padded = qt.shape[1]
    _expect_all([(x, "x", (T, C), _HI), (offsets, "offsets", (E + 1,), _I64), (q, "q", (T, C), _U8),
                 (s, "s", (C // 128, T), _F32), (qt, "qt", (C, padded), _U8),
                 (st, "st", (padded // 128, C), _F32)])
    return (_ptr(x), _in_type(x), T, C, _ld(x), _ptr(offsets), E, fmt_rows, _ptr(q), _ld(q) if q is not None else 0,
            _ptr(s), _ld(s) if s is not None else 0, fmt_cols, _ptr(qt), _ld(qt), _ptr(st), _ld(st), padded, _stream(x))


@_entry
def fp8bq_grouped_gemm_fprop(qx, sx, fx, offsets, qw, sw, fw, y):
    T, K = qx.shape
    E = _experts(offsets)
    N = _stacked(qw.shape[0], E, "qw")
    _expect_all([(qx, "qx", (T, K), _U8), (sx, "sx", (K // 128, T), _F32), (offsets, "offsets", (E + 1,), _I64),
                 (qw, "qw", (E * N, K), _U8), (sw, "sw", (E * N // 128, K // 128), _F32), (y, "y", (T, N), _HI)])
    return (E, T, N, K, _ptr(offsets), _ptr(qx), _ld(qx), _ptr(sx), _ld(sx), fx, _ptr(qw), _ld(qw), _ptr(sw), _ld(sw),
            fw, _ptr(y), _out_type(y), _ld(y), _stream(y))


@_entry
def fp8bq_grouped_gemm_dgrad(qdy, sdy, fdy, offsets, qwt, sw, fw, dx):
    T, N = qdy.shape
    E = _experts(offsets)
    K = qwt.shape[0]
    _expect_all([(qdy, "qdy", (T, N), _U8), (sdy, "sdy", (N // 128, T), _F32), (offsets, "offsets", (E + 1,), _I64),
                 (qwt, "qwt", (K, E * N), _U8), (sw, "sw", (E * N // 128, K // 128), _F32), (dx, "dx", (T, K), _HI)])
    return (E, T, N, K, _ptr(offsets), _ptr(qdy), _ld(qdy), _ptr(sdy), _ld(sdy), fdy, _ptr(qwt), _ld(qwt), _ptr(sw),
            _ld(sw), fw, _ptr(dx), _out_type(dx), _ld(dx), _stream(dx))


@_entry
def fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fdy, qxt, sxt, fx, offsets, dw, accumulate=False):
    N, padded = qdyt.shape
    E = _experts(offsets)
    K = qxt.shape[0]
    _expect_all([(qdyt, "qdyt", (N, padded), _U8), (sdyt, "sdyt", (padded // 128, N), _F32),
                 (qxt, "qxt", (K, padded), _U8), (sxt, "sxt", (padded // 128, K), _F32),
                 (offsets, "offsets", (E + 1,), _I64), (dw, "dw", (E * N, K), _F32 if accumulate else _HI)])
    return (E, padded, N, K, _ptr(offsets), _ptr(qdyt), _ld(qdyt), _ptr(sdyt), _ld(sdyt), fdy, _ptr(qxt), _ld(qxt),
            _ptr(sxt), _ld(sxt), fx, _ptr(dw), OUT_F32_ACCUM if accumulate else _out_type(dw), _ld(dw), _stream(dw))


def _cols_outputs(x, offsets):
    T, C = x.shape
    padded = fp8bq_grouped_padded_rows(T, _experts(offsets))
    qt = torch.empty((C, padded), dtype=torch.uint8, device=x.device)
    return qt, torch.empty((padded // 128, C), dtype=torch.float32, device=x.device)


def quantize_act_grouped_128x1(x, offsets, fmt=E4M3):
    qt, st = _cols_outputs(x, offsets)
    fp8bq_quantize_act_grouped(x, offsets, E4M3, None, None, fmt, qt, st)
    return qt, st


def quantize_act_grouped_dual(x, offsets, fmt_rows=E4M3, fmt_cols=E4M3):
    """(q, s) of quantize_act_1x128(x, fmt_rows) and (qt, st) of quantize_act_grouped_128x1(x, offsets,
    fmt_cols) from one pass over x."""
    T, C = x.shape
    q = torch.empty((T, C), dtype=torch.uint8, device=x.device)
    s = torch.empty((C // 128, _pad4(T)), dtype=torch.float32, device=x.device)[:, :T]
    qt, st = _cols_outputs(x, offsets)
    fp8bq_quantize_act_grouped(x, offsets, fmt_rows, q, s, fmt_cols, qt, st)
    return q, s, qt, st


def grouped_gemm_fprop(qx, sx, offsets, qw, sw, fx=E4M3, fw=E4M3, out_dtype=torch.bfloat16, out=None):
    N = _stacked(qw.shape[0], _experts(offsets), "qw")
    y = out if out is not None else torch.empty((qx.shape[0], N), dtype=out_dtype, device=qx.device)
    fp8bq_grouped_gemm_fprop(qx, sx, fx, offsets, qw, sw, fw, y)
    return y


def grouped_gemm_dgrad(qdy, sdy, offsets, qwt, sw, fdy=E4M3, fw=E4M3, out_dtype=torch.bfloat16, out=None):
    dx = out if out is not None else torch.empty((qdy.shape[0], qwt.shape[0]), dtype=out_dtype, device=qdy.device)
    fp8bq_grouped_gemm_dgrad(qdy, sdy, fdy, offsets, qwt, sw, fw, dx)
    return dx


def grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offsets, fdy=E4M3, fx=E4M3, out_dtype=torch.bfloat16, out=None,
                       accumulate=False):
    """accumulate=True adds the result to `out` (an FP32 main-grad buffer) instead of overwriting it."""
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate=True needs an FP32 `out` tensor holding the running sum")
    dw = out if out is not None else torch.empty((_experts(offsets) * qdyt.shape[0], qxt.shape[0]), dtype=out_dtype,
                                                 device=qdyt.device)
    fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fdy, qxt, sxt, fx, offsets, dw, accumulate=accumulate)
    return dw
