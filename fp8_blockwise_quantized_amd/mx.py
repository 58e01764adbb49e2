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

import torch

from . import (_HI, _U8, OUT_F32_ACCUM, _c_i64, _c_int, _c_sz, _c_vp, _entry, _expect_all, _F32, _in_type, _ld,
               _out_type, _ptr, _RESTYPES, _SIGS, _stream, _ws_args, lib)
from .grouped import _I64, _experts, _stacked

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


def _lds(s):
    """Leading dimension, in words, of scales [words, R, 4]."""
    if s.numel() == 0:
        return max(s.size(1), 1)
    if s.stride(2) != 1 or (s.size(1) > 1 and s.stride(1) != 4) or (s.size(0) > 1 and s.stride(0) % 4):
        raise ValueError("scales must be [words, rows, 4] with rows of four bytes next to each other")
    return s.stride(0) // 4 if s.size(0) > 1 else s.size(1)


def _ldo(t):
    """Leading dimension of an output (any, even where one row leaves it undefined)."""
    return max(_ld(t), t.size(1), 1)


def _words(n):
    return (n + 127) // 128


@_entry
def fp8bq_quantize_mxfp4(x, q, s, qt, st):
    R, C = x.shape
    _expect_all([(x, "x", (R, C), _HI), (q, "q", (R, C // 2), _U8), (s, "s", (_words(C), R, 4), _U8),
                 (qt, "qt", (C, (R + 31) // 32 * 16), _U8), (st, "st", (_words(R), C, 4), _U8)])
    return (_ptr(x), _in_type(x), R, C, _ld(x), _ptr(q), _ld(q) if q is not None else 0, _ptr(s),
            _lds(s) if s is not None else 0, _ptr(qt), _ld(qt) if qt is not None else 0, _ptr(st),
            _lds(st) if st is not None else 0, _stream(x))


@_entry
def fp8bq_gemm_mxfp4(qa, sa, qb, sb, c, ws=None, accumulate=False):
    M, K = qa.shape[0], 2 * qa.shape[1]
    N = qb.shape[0]
    _expect_all([(qa, "qa", (M, K // 2), _U8), (sa, "sa", (_words(K), M, 4), _U8), (qb, "qb", (N, K // 2), _U8),
                 (sb, "sb", (_words(K), N, 4), _U8), (c, "c", (M, N), _F32 if accumulate else _HI)], ws)
    wsp, wsb = _ws_args(ws)
    return (M, N, K, _ptr(qa), _ld(qa), _ptr(sa), _lds(sa), _ptr(qb), _ld(qb), _ptr(sb), _lds(sb), _ptr(c),
            OUT_F32_ACCUM if accumulate else _out_type(c), _ldo(c), wsp, wsb, _stream(c))


@_entry
def fp8bq_linear_mxfp4(x, qw, sw, y, ws=None):
    M, K = x.shape
    N = qw.shape[0]
    _expect_all([(x, "x", (M, K), _HI), (qw, "qw", (N, K // 2), _U8), (sw, "sw", (_words(K), N, 4), _U8),
                 (y, "y", (M, N), _HI)], ws)
    wsp, wsb = _ws_args(ws)
    return (M, N, K, _ptr(x), _in_type(x), _ld(x), _ptr(qw), _ld(qw), _ptr(sw), _lds(sw), _ptr(y), _out_type(y),
            _ldo(y), wsp, wsb, _stream(y))


@_entry
def fp8bq_grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, y, ws=None):
    T, K = qa.shape[0], 2 * qa.shape[1]
    E = _experts(offsets)
    N = _stacked(qw.shape[0], E, "qw")
    _expect_all([(qa, "qa", (T, K // 2), _U8), (sa, "sa", (_words(K), T, 4), _U8), (offsets, "offsets", (E + 1,), _I64),
                 (qw, "qw", (E * N, K // 2), _U8), (sw, "sw", (_words(K), E * N, 4), _U8), (y, "y", (T, N), _HI)], ws)
    wsp, wsb = _ws_args(ws)
    return (E, T, N, K, _ptr(offsets), _ptr(qa), _ld(qa), _ptr(sa), _lds(sa), _ptr(qw), _ld(qw), _ptr(sw), _lds(sw),
            _ptr(y), _out_type(y), _ldo(y), wsp, wsb, _stream(y))


@_entry
def fp8bq_grouped_linear_mxfp4(x, offsets, qw, sw, y, ws=None):
    T, K = x.shape
    E = _experts(offsets)
    N = _stacked(qw.shape[0], E, "qw")
    _expect_all([(x, "x", (T, K), _HI), (offsets, "offsets", (E + 1,), _I64), (qw, "qw", (E * N, K // 2), _U8),
                 (sw, "sw", (_words(K), E * N, 4), _U8), (y, "y", (T, N), _HI)], ws)
    wsp, wsb = _ws_args(ws)
    return (E, T, N, K, _ptr(offsets), _ptr(x), _in_type(x), _ld(x), _ptr(qw), _ld(qw), _ptr(sw), _lds(sw), _ptr(y),
            _out_type(y), _ldo(y), wsp, wsb, _stream(y))


def _codes(R, K, device):
    return (torch.empty((R, K // 2), dtype=torch.uint8, device=device),
            torch.empty((_words(K), R, 4), dtype=torch.uint8, device=device))


def quantize_mxfp4(x):
    q, s = _codes(*x.shape, x.device)
    fp8bq_quantize_mxfp4(x, q, s, None, None)
    return q, s


def quantize_mxfp4_t(x):
    R, C = x.shape
    qt, st = _codes(C, (R + 31) // 32 * 32, x.device)
    fp8bq_quantize_mxfp4(x, None, None, qt, st)
    return qt, st


def quantize_mxfp4_dual(x):
    R, C = x.shape
    q, s = _codes(R, C, x.device)
    qt, st = _codes(C, (R + 31) // 32 * 32, x.device)
    fp8bq_quantize_mxfp4(x, q, s, qt, st)
    return q, s, qt, st


def _space(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _output(out, M, N, dtype, like):
    return out if out is not None else torch.empty((M, N), dtype=dtype, device=like.device)


def gemm_mxfp4(qa, sa, qb, sb, out_dtype=torch.bfloat16, out=None, ws=None, accumulate=False):
    """accumulate=True adds the result to `out` (FP32) instead of overwriting it."""
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate=True needs an FP32 `out` tensor holding the running sum")
    M, K2 = qa.shape
    N = qb.shape[0]
    c = _output(out, M, N, out_dtype, qa)
    if ws is None:
        ws = _space(fp8bq_gemm_mxfp4_workspace_size(M, N, 2 * K2), qa.device)
    fp8bq_gemm_mxfp4(qa, sa, qb, sb, c, ws, accumulate=accumulate)
    return c


def linear_mxfp4(x, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    M, K = x.shape
    N = qw.shape[0]
    y = _output(out, M, N, out_dtype, x)
    if ws is None:
        ws = _space(fp8bq_linear_mxfp4_workspace_size(M, N, K), x.device)
    fp8bq_linear_mxfp4(x, qw, sw, y, ws)
    return y


def grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    T, K2 = qa.shape
    E = _experts(offsets)
    N = _stacked(qw.shape[0], E, "qw")
    y = _output(out, T, N, out_dtype, qa)
    if ws is None:
        ws = _space(fp8bq_grouped_gemm_mxfp4_workspace_size(E, T, N, 2 * K2), qa.device)
    fp8bq_grouped_gemm_mxfp4(qa, sa, offsets, qw, sw, y, ws)
    return y


def grouped_linear_mxfp4(x, offsets, qw, sw, out_dtype=torch.bfloat16, out=None, ws=None):
    T, K = x.shape
    E = _experts(offsets)
    N = _stacked(qw.shape[0], E, "qw")
    y = _output(out, T, N, out_dtype, x)
    if ws is None:
        ws = _space(fp8bq_grouped_linear_mxfp4_workspace_size(E, T, N, K), x.device)
    fp8bq_grouped_linear_mxfp4(x, offsets, qw, sw, y, ws)
    return y
