"""Orthogonalization of updates by Newton-Schulz products (binding of include/fp8bq_ortho.h).

Raw entry point, tensors in place of pointers:

    fp8bq_orthogonalize(g, coefficients, eps, out, ws)     coefficients: (a, b, c) of every step
    fp8bq_orthogonalize_workspace_size(B, R, C)

Allocating helper:

    orthogonalize(g, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out=None, ws=None)
        -> BF16 of g's shape; g [R, C] or [B, R, C], BF16 or FP32.  coefficients: one (a, b, c) for all steps or a list
        of one for each.

An optimizer step that moves a matrix along its orthogonalized momentum and keeps it at a fixed radius:
hyperball_step(w, orthogonalize(momentum), lr, weight_decay, radius=r).
"""

import ctypes

import torch

from . import IN_BF16, IN_F32, _RESTYPES, _SIGS, _c_i64, _c_int, _c_sz, _c_vp, _entry, lib
from ._marshal import BF16, HI, batch, on_its_device, space, stream
from .mx import _space

MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)

_SIGS.update({
    "fp8bq_orthogonalize": [_c_vp, _c_int] + [_c_i64] * 5 + [ctypes.c_int32, _c_vp, ctypes.c_double, _c_vp, _c_i64, _c_i64,
                                                             _c_vp, _c_sz, _c_vp],
    "fp8bq_orthogonalize_workspace_size": [_c_i64] * 3,
})
_RESTYPES["fp8bq_orthogonalize_workspace_size"] = _c_sz


def fp8bq_orthogonalize_workspace_size(B, R, C):
    return lib().fp8bq_orthogonalize_workspace_size(B, R, C)


def _steps(coefficients):
    rows = [tuple(float(v) for v in row) for row in coefficients]
    if any(len(row) != 3 for row in rows):
        raise ValueError("coefficients: three of each step")
    return (ctypes.c_double * (3 * len(rows)))(*[v for row in rows for v in row])


@on_its_device
@_entry
def fp8bq_orthogonalize(g, coefficients, eps, out, ws):
    if not isinstance(g, torch.Tensor) or g.dim() not in (2, 3):
        raise ValueError("g must be a matrix or a batch of matrices")
    dev = g.get_device()
    gp, B, R, C, ldg, gstride = batch(g, "g", g.shape, HI, dev)
    op, _, _, _, ldo, ostride = batch(out, "out", g.shape, BF16, dev)
    steps = _steps(coefficients)
    wsp, wsb = space(ws, dev)
    return (gp, IN_BF16 if g.dtype == torch.bfloat16 else IN_F32, B, R, C, ldg, gstride, len(steps) // 3, steps, float(eps), op,
            ldo, ostride, wsp, wsb, stream(dev))


@on_its_device
def orthogonalize(g, steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7, out=None, ws=None):
    if not isinstance(coefficients[0], (tuple, list)):
        coefficients = [coefficients] * steps
    elif len(coefficients) != steps:
        raise ValueError(f"{len(coefficients)} steps' coefficients for {steps} steps")
    if out is None:
        out = g.new_empty(g.shape, dtype=torch.bfloat16)
    if ws is None:
        B, R, C = g.shape if g.dim() == 3 else (1, *g.shape)
        ws = _space("fp8bq_orthogonalize_workspace_size", g, B, R, C)
    fp8bq_orthogonalize.__wrapped__(g, coefficients, eps, out, ws)
    return out
