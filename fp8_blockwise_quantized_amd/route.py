"""Routing of tokens to experts and the experts' rows (binding of include/fp8bq_route.h).

Raw entry points, tensors in place of pointers:

    fp8bq_route_experts(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale, experts, weights)
    fp8bq_route_experts_backward(dweights, logits, score, renormalize, scale, experts, dlogits)
    fp8bq_expert_rows(experts, E, offsets, rows, slots, ws=None)
    fp8bq_expert_rows_workspace_size(n, E)
    fp8bq_gather_rows(x, slots, k, out)
    fp8bq_combine_rows(y, rows, weights, out)
    fp8bq_combine_rows_backward(dout, y, rows, weights, slots, dy, dweights)

Allocating helpers (score: "softmax" or "sigmoid"):

    route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True,
                  scale=1.0) -> (experts [T, k] int32, weights [T, k] float32)
    route_experts_backward(dweights, logits, experts, score="softmax", renormalize=True, scale=1.0) -> dlogits [T, E]
    expert_rows(experts, E) -> (offsets [E + 1] int64, rows [T, k] int32, slots [T k] int32)
    gather_rows(x, slots, k) -> [T k, H] in the experts' order
    combine_rows(y, rows, weights=None, out_dtype=None) -> [T, H]
    combine_rows_backward(dout, y, rows, weights, slots) -> (dy [T k, H], dweights [T, k])

A mixture-of-experts layer: experts, w = route_experts(x @ router, k); offsets, rows, slots = expert_rows(experts, E);
xs = gather_rows(x, slots, k); the grouped products on xs and offsets give y; out = combine_rows(y, rows, w).  Backward:
dy, dw = combine_rows_backward(dout, y, rows, w, slots); the grouped products give dxs; dx = combine_rows(dxs, rows) plus
what comes through route_experts_backward(dw, logits, experts).
"""

import ctypes

import torch

from . import (Fp8bqError, IN_BF16, IN_F32, OUT_BF16, OUT_F32, _RESTYPES, _SIGS, _c_i64, _c_int, _c_sz, _c_vp, _entry,
               lib)
from ._marshal import F32, HI, I32, I64, flat, matrix, on_its_device, space, stream, vector
from .mx import _space

MAX_CHOICES = 64
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}

_c_f64 = ctypes.c_double
_SIGS.update({
    "fp8bq_route_experts": [_c_vp, _c_int] + [_c_i64] * 4 + [_c_int, _c_vp] + [_c_i64] * 3 + [_c_int, _c_f64] + [_c_vp] * 3,
    "fp8bq_route_experts_backward": [_c_vp, _c_vp, _c_int] + [_c_i64] * 4 + [_c_int, _c_int, _c_f64, _c_vp, _c_vp, _c_i64,
                                                                           _c_vp],
    "fp8bq_expert_rows_workspace_size": [_c_i64] * 2,
    "fp8bq_expert_rows": [_c_vp, _c_i64, _c_i64] + [_c_vp] * 4 + [_c_sz, _c_vp],
    "fp8bq_gather_rows": [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp],
    "fp8bq_combine_rows": [_c_vp, _c_int] + [_c_i64] * 4 + [_c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_vp],
    "fp8bq_combine_rows_backward": [_c_vp, _c_int, _c_i64] * 2 + [_c_i64] * 3 + [_c_vp] * 4 + [_c_i64, _c_vp, _c_vp],
})
_RESTYPES["fp8bq_expert_rows_workspace_size"] = _c_sz


def fp8bq_expert_rows_workspace_size(n, E):
    return lib().fp8bq_expert_rows_workspace_size(n, E)


def _in(t):
    return IN_BF16 if t.dtype == torch.bfloat16 else IN_F32


def _k_of(t, name):
    """k of a [T, k] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have shape [T, k], not {tuple(t.shape)}")
    return t.shape[1]


def _call(name, *args):
    status = getattr(lib(), name)(*args)
    if status != 0:
        raise Fp8bqError(status, name)


# (what an entry point needs beside its outputs' addresses, so that the helpers need not check what they have made)
def _route(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale, dev):
    T, E = logits.shape
    xp, ldx = matrix(logits, "logits", (T, E), HI, dev)
    bp = vector(bias, "bias", E, F32, dev) if bias is not None else 0
    return xp, _in(logits), T, E, ldx, k, score, bp, groups, top_groups, group_best, 1 if renormalize else 0, float(scale)


def _route_backward(dweights, logits, score, renormalize, scale, experts, dev):
    T, E = logits.shape
    k = _k_of(experts, "experts")
    dwp = flat(dweights, "dweights", (T, k), F32, dev)
    xp, ldx = matrix(logits, "logits", (T, E), HI, dev)
    ep = flat(experts, "experts", (T, k), I32, dev)
    return dwp, xp, _in(logits), T, E, ldx, k, score, 1 if renormalize else 0, float(scale), ep


def _gather(x, slots, k, dev):
    T, H = x.shape
    xp, ldx = matrix(x, "x", (T, H), HI, dev)
    return xp, _in(x), T, H, ldx, vector(slots, "slots", T * k, I32, dev), k


def _combine(y, rows, weights, dev):
    k = _k_of(rows, "rows")
    T, H = rows.shape[0], y.shape[1]
    yp, ldy = matrix(y, "y", (T * k, H), HI, dev)
    rp = flat(rows, "rows", (T, k), I32, dev)
    return yp, _in(y), T, k, H, ldy, rp, flat(weights, "weights", (T, k), F32, dev) if weights is not None else 0


def _combine_backward(dout, y, rows, weights, slots, dev):
    T, H = dout.shape
    k = _k_of(rows, "rows")
    dp, lddo = matrix(dout, "dout", (T, H), HI, dev)
    yp, ldy = matrix(y, "y", (T * k, H), HI, dev)
    rp, wp = flat(rows, "rows", (T, k), I32, dev), flat(weights, "weights", (T, k), F32, dev)
    return dp, _in(dout), lddo, yp, _in(y), ldy, T, k, H, rp, wp, vector(slots, "slots", T * k, I32, dev)


@on_its_device
@_entry
def fp8bq_route_experts(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale, experts, weights):
    dev = logits.get_device()
    args = _route(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale, dev)
    shape = (logits.shape[0], k)
    return (*args, flat(experts, "experts", shape, I32, dev), flat(weights, "weights", shape, F32, dev), stream(dev))


@on_its_device
@_entry
def fp8bq_route_experts_backward(dweights, logits, score, renormalize, scale, experts, dlogits):
    dev = logits.get_device()
    args = _route_backward(dweights, logits, score, renormalize, scale, experts, dev)
    dp, ldd = matrix(dlogits, "dlogits", logits.shape, (logits.dtype,), dev)
    return (*args, dp, ldd, stream(dev))


@on_its_device
@_entry
def fp8bq_expert_rows(experts, E, offsets, rows, slots, ws=None):
    dev = experts.get_device()
    shape, n = (experts.shape[0], _k_of(experts, "experts")), experts.numel()
    ep = flat(experts, "experts", shape, I32, dev)
    op, rp = vector(offsets, "offsets", E + 1, I64, dev), flat(rows, "rows", shape, I32, dev)
    sp = vector(slots, "slots", n, I32, dev)
    wsp, wsb = space(ws, dev)
    return ep, n, E, op, rp, sp, wsp, wsb, stream(dev)


@on_its_device
@_entry
def fp8bq_gather_rows(x, slots, k, out):
    dev = x.get_device()
    args = _gather(x, slots, k, dev)
    op, ldo = matrix(out, "out", (x.shape[0] * k, x.shape[1]), (x.dtype,), dev)
    return (*args, op, ldo, stream(dev))


@on_its_device
@_entry
def fp8bq_combine_rows(y, rows, weights, out):
    dev = y.get_device()
    args = _combine(y, rows, weights, dev)
    op, ldo = matrix(out, "out", (rows.shape[0], y.shape[1]), HI, dev)
    return (*args, op, OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32, ldo, stream(dev))


@on_its_device
@_entry
def fp8bq_combine_rows_backward(dout, y, rows, weights, slots, dy, dweights):
    dev = dout.get_device()
    args = _combine_backward(dout, y, rows, weights, slots, dev)
    gp, ldg = matrix(dy, "dy", y.shape, (y.dtype,), dev)
    return (*args, gp, ldg, flat(dweights, "dweights", weights.shape, F32, dev), stream(dev))


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    return _SCORES[score]


@on_its_device
def route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    dev = logits.get_device()
    args = _route(logits, k, _score(score), bias, groups, top_groups, group_best, renormalize, scale, dev)
    at = stream(dev)
    shape = (logits.shape[0], k)
    experts, weights = logits.new_empty(shape, dtype=torch.int32), logits.new_empty(shape, dtype=torch.float32)
    _call("fp8bq_route_experts", *args, experts.data_ptr(), weights.data_ptr(), at)
    return experts, weights


@on_its_device
def route_experts_backward(dweights, logits, experts, score="softmax", renormalize=True, scale=1.0):
    dev = logits.get_device()
    args = _route_backward(dweights, logits, _score(score), renormalize, scale, experts, dev)
    at = stream(dev)
    dlogits = logits.new_empty(logits.shape)
    _call("fp8bq_route_experts_backward", *args, dlogits.data_ptr(), max(logits.shape[1], 1), at)
    return dlogits


@on_its_device
def expert_rows(experts, E):
    dev = experts.get_device()
    shape, n = (experts.shape[0], _k_of(experts, "experts")), experts.numel()
    ep = flat(experts, "experts", shape, I32, dev)
    at = stream(dev)
    offsets = experts.new_empty(E + 1, dtype=torch.int64)
    rows, slots = experts.new_empty(shape), experts.new_empty(n)
    ws = _space("fp8bq_expert_rows_workspace_size", experts, n, E)
    wsp, wsb = (0, 0) if ws is None else (ws.data_ptr(), ws.numel())
    _call("fp8bq_expert_rows", ep, n, E, offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), wsp, wsb, at)
    return offsets, rows, slots


@on_its_device
def gather_rows(x, slots, k):
    dev = x.get_device()
    args = _gather(x, slots, k, dev)
    at = stream(dev)
    T, H = x.shape
    out = x.new_empty((T * k, H))
    _call("fp8bq_gather_rows", *args, out.data_ptr(), H, at)
    return out


@on_its_device
def combine_rows(y, rows, weights=None, out_dtype=None):
    """out_dtype: y's, or bfloat16 or float32."""
    dev = y.get_device()
    args = _combine(y, rows, weights, dev)
    if out_dtype is None:
        out_dtype = y.dtype
    elif out_dtype not in HI:
        raise TypeError(f"out_dtype must be bfloat16 or float32, not {out_dtype}")
    at = stream(dev)
    H = y.shape[1]
    out = y.new_empty((rows.shape[0], H), dtype=out_dtype)
    _call("fp8bq_combine_rows", *args, out.data_ptr(), OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32, H, at)
    return out


@on_its_device
def combine_rows_backward(dout, y, rows, weights, slots):
    dev = dout.get_device()
    args = _combine_backward(dout, y, rows, weights, slots, dev)
    at = stream(dev)
    # (the call writes nothing where the rows have no elements)
    dy, dweights = y.new_empty(y.shape), weights.new_empty(weights.shape) if y.shape[1] else weights.new_zeros(weights.shape)
    _call("fp8bq_combine_rows_backward", *args, dy.data_ptr(), y.shape[1], dweights.data_ptr(), at)
    return dy, dweights
