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

from . import IN_BF16, IN_F32, OUT_BF16, OUT_F32, _RESTYPES, _SIGS, _c_i64, _c_int, _c_sz, _c_vp, _entry, lib
from ._marshal import F32, HI, I32, I64, matrix, on_its_device, space, stream, vector
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


def _choices(t, name, T, dtypes, dev):
    """Address and k of a contiguous [T, k] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 2 or t.shape[0] != T:
        raise ValueError(f"{name} must have shape [{T}, k], not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return vector(t.view(-1), name, t.numel(), dtypes, dev), t.shape[1]


def _same(t, name, T, k, dtypes, dev):
    p, n = _choices(t, name, T, dtypes, dev)
    if n != k:
        raise ValueError(f"{name} must have shape [{T}, {k}], not {tuple(t.shape)}")
    return p


@on_its_device
@_entry
def fp8bq_route_experts(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale, experts, weights):
    T, E = logits.shape
    dev = logits.get_device()
    xp, ldx = matrix(logits, "logits", (T, E), HI, dev)
    bp = vector(bias, "bias", E, F32, dev) if bias is not None else 0
    ep, wp = _same(experts, "experts", T, k, I32, dev), _same(weights, "weights", T, k, F32, dev)
    return (xp, _in(logits), T, E, ldx, k, score, bp, groups, top_groups, group_best, int(bool(renormalize)), float(scale),
            ep, wp, stream(dev))


@on_its_device
@_entry
def fp8bq_route_experts_backward(dweights, logits, score, renormalize, scale, experts, dlogits):
    T, E = logits.shape
    dev = dweights.get_device()
    dwp, k = _choices(dweights, "dweights", T, F32, dev)
    xp, ldx = matrix(logits, "logits", (T, E), HI, dev)
    ep = _same(experts, "experts", T, k, I32, dev)
    dp, ldd = matrix(dlogits, "dlogits", (T, E), (logits.dtype,), dev)
    return dwp, xp, _in(logits), T, E, ldx, k, score, int(bool(renormalize)), float(scale), ep, dp, ldd, stream(dev)


@on_its_device
@_entry
def fp8bq_expert_rows(experts, E, offsets, rows, slots, ws=None):
    dev = experts.get_device()
    ep, k = _choices(experts, "experts", experts.shape[0], I32, dev)
    n = experts.numel()
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch tensor")
    op = vector(offsets, "offsets", E + 1, I64, dev)
    rp = _same(rows, "rows", experts.shape[0], k, I32, dev)
    sp = vector(slots, "slots", n, I32, dev)
    wsp, wsb = space(ws, dev)
    return ep, n, E, op, rp, sp, wsp, wsb, stream(dev)


@on_its_device
@_entry
def fp8bq_gather_rows(x, slots, k, out):
    T, H = x.shape
    dev = x.get_device()
    xp, ldx = matrix(x, "x", (T, H), HI, dev)
    sp = vector(slots, "slots", T * k, I32, dev)
    op, ldo = matrix(out, "out", (T * k, H), (x.dtype,), dev)
    return xp, _in(x), T, H, ldx, sp, k, op, ldo, stream(dev)


@on_its_device
@_entry
def fp8bq_combine_rows(y, rows, weights, out):
    T = rows.shape[0]
    dev = y.get_device()
    rp, k = _choices(rows, "rows", T, I32, dev)
    H = y.shape[1]
    yp, ldy = matrix(y, "y", (T * k, H), HI, dev)
    wp = _same(weights, "weights", T, k, F32, dev) if weights is not None else 0
    op, ldo = matrix(out, "out", (T, H), HI, dev)
    return (yp, _in(y), T, k, H, ldy, rp, wp, op, OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32, ldo, stream(dev))


@on_its_device
@_entry
def fp8bq_combine_rows_backward(dout, y, rows, weights, slots, dy, dweights):
    T, H = dout.shape
    dev = dout.get_device()
    dp, lddo = matrix(dout, "dout", (T, H), HI, dev)
    rp, k = _choices(rows, "rows", T, I32, dev)
    yp, ldy = matrix(y, "y", (T * k, H), HI, dev)
    wp = _same(weights, "weights", T, k, F32, dev)
    sp = vector(slots, "slots", T * k, I32, dev)
    gp, ldg = matrix(dy, "dy", (T * k, H), (y.dtype,), dev)
    dwp = _same(dweights, "dweights", T, k, F32, dev)
    return dp, _in(dout), lddo, yp, _in(y), ldy, T, k, H, rp, wp, sp, gp, ldg, dwp, stream(dev)


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    return _SCORES[score]


def route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    T = logits.shape[0]
    experts, weights = logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k), dtype=torch.float32)
    fp8bq_route_experts(logits, k, _score(score), bias, groups, top_groups, group_best, renormalize, scale, experts, weights)
    return experts, weights


def route_experts_backward(dweights, logits, experts, score="softmax", renormalize=True, scale=1.0):
    dlogits = logits.new_empty(logits.shape)
    fp8bq_route_experts_backward(dweights, logits, _score(score), renormalize, scale, experts, dlogits)
    return dlogits


@on_its_device
def expert_rows(experts, E):
    n = experts.numel()
    offsets = experts.new_empty(E + 1, dtype=torch.int64)
    rows, slots = experts.new_empty(experts.shape), experts.new_empty(n)
    fp8bq_expert_rows(experts, E, offsets, rows, slots, _space("fp8bq_expert_rows_workspace_size", experts, n, E))
    return offsets, rows, slots


def gather_rows(x, slots, k):
    out = x.new_empty((x.shape[0] * k, x.shape[1]))
    fp8bq_gather_rows(x, slots, k, out)
    return out


def combine_rows(y, rows, weights=None, out_dtype=None):
    """out_dtype: y's, or bfloat16 or float32."""
    out = y.new_empty((rows.shape[0], y.shape[1]), dtype=out_dtype or y.dtype)
    fp8bq_combine_rows(y, rows, weights, out)
    return out


def combine_rows_backward(dout, y, rows, weights, slots):
    dy, dweights = y.new_empty(y.shape), weights.new_empty(weights.shape)
    fp8bq_combine_rows_backward(dout, y, rows, weights, slots, dy, dweights)
    return dy, dweights
