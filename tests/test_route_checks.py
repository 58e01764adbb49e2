"""Refusals of the routing entry points, without a GPU: the C ABI's statuses on fake pointers and the Python binding's
checks."""

import ctypes
import os
import re

import pytest
import torch

import fp8_blockwise_quantized_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, LD, ALIGN, DTYPE, FORMAT, WORKSPACE, DEVICE, LAUNCH, OVERLAP, VALUE = range(12)
HAVE_GPU = torch.cuda.is_available()
P = lambda i, plus=0: ctypes.c_void_p(0x10000000 * (i + 1) + plus)
NUL = ctypes.c_void_p(0)
T, E, K, H = 100, 64, 6, 128
BIG = 1 << 40


def route(x=P(0), xt=1, T=T, E=E, ldx=E, k=K, score=0, bias=P(1), groups=4, top=2, best=2, renorm=1, scale=1.0, e=P(2), w=P(3)):
    return fq.lib().fp8bq_route_experts(x, xt, T, E, ldx, k, score, bias, groups, top, best, renorm, scale, e, w, NUL)


def back(dw=P(1), x=P(0), xt=1, T=T, E=E, ldx=E, k=K, score=0, renorm=1, scale=1.0, e=P(2), dx=P(3), lddx=E):
    return fq.lib().fp8bq_route_experts_backward(dw, x, xt, T, E, ldx, k, score, renorm, scale, e, dx, lddx, NUL)


def rows(e=P(0), n=5000, E=E, off=P(1), r=P(2), s=P(3), ws=P(4), wsb=BIG):
    return fq.lib().fp8bq_expert_rows(e, n, E, off, r, s, ws, wsb, NUL)


def gather(x=P(0), xt=0, T=T, H=H, ldx=H, s=P(1), k=K, out=P(2), ldo=H):
    return fq.lib().fp8bq_gather_rows(x, xt, T, H, ldx, s, k, out, ldo, NUL)


def combine(y=P(0), yt=0, T=T, k=K, H=H, ldy=H, r=P(1), w=P(2), out=P(3), ot=0, ldo=H):
    return fq.lib().fp8bq_combine_rows(y, yt, T, k, H, ldy, r, w, out, ot, ldo, NUL)


def combine_back(d=P(0), dt=0, ldd=H, y=P(1), yt=0, ldy=H, T=T, k=K, H=H, r=P(2), w=P(3), s=P(4), dy=P(5), ldg=H, dw=P(6)):
    return fq.lib().fp8bq_combine_rows_backward(d, dt, ldd, y, yt, ldy, T, k, H, r, w, s, dy, ldg, dw, NUL)


ALL = (route, back, rows, gather, combine, combine_back)


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bq_route.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp8bq_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 7
    for n in names:
        assert hasattr(fq, n) and hasattr(fq.lib(), n), n


@pytest.mark.skipif(HAVE_GPU, reason="fake pointers: checks the no-device path")
def test_valid_arguments_reach_the_device_check():
    for f in ALL:
        assert f() == DEVICE, f
    assert route(bias=NUL, groups=1, top=1, best=1, k=64) == route(x=P(0, 4), ldx=E + 1) == DEVICE
    assert back(x=P(0, 4), ldx=E + 1, lddx=E + 3) == combine(w=NUL, ot=1) == rows(n=0) == DEVICE
    assert rows(n=100, ws=NUL, wsb=0) == combine_back(dt=1, yt=1) == DEVICE


def test_empty_calls_succeed():
    assert route(T=0) == back(T=0) == gather(T=0) == combine(T=0) == combine_back(T=0) == OK
    assert gather(H=0) == combine(H=0) == combine_back(H=0) == OK


def test_route_refusals():
    for f in (route, back):
        assert f(xt=2) == DTYPE and f(score=2) == f(scale=float("nan")) == f(scale=float("inf")) == VALUE
        assert f(T=-1) == f(E=0) == f(E=513, ldx=513) == f(k=0) == f(k=65) == f(T=1 << 30) == SHAPE
        assert f(x=NUL) == f(e=NUL) == NULL
        assert f(x=P(0, 2)) == f(e=P(2, 2)) == ALIGN
        assert f(ldx=E - 1) == LD
    assert route(k=33) == route(groups=3) == route(groups=0) == route(top=0) == route(top=5) == route(best=0) == SHAPE
    assert route(best=3) == route(groups=64, top=8, best=2) == route(groups=65, E=130, ldx=130, best=1) == SHAPE
    assert route(w=NUL) == back(dw=NUL) == back(dx=NUL) == NULL
    assert route(bias=P(1, 2)) == route(w=P(3, 1)) == back(dw=P(1, 2)) == back(dx=P(3, 2)) == ALIGN
    assert back(lddx=E - 1) == LD
    assert route(e=P(0)) == route(w=P(0)) == route(e=P(1)) == route(w=P(2)) == OVERLAP
    assert back(dx=P(0)) == back(dx=P(1)) == back(dx=P(2)) == OVERLAP


def test_rows_refusals():
    assert rows(n=-1) == rows(n=1 << 31) == rows(E=0) == rows(E=513) == SHAPE
    assert rows(e=NUL) == rows(off=NUL) == rows(r=NUL) == rows(s=NUL) == rows(n=0, off=NUL) == NULL
    assert rows(e=P(0, 2)) == rows(off=P(1, 4)) == rows(r=P(2, 1)) == rows(s=P(3, 2)) == rows(ws=P(4, 8)) == ALIGN
    assert rows(off=P(0)) == rows(r=P(0)) == rows(s=P(2)) == rows(ws=P(3)) == OVERLAP
    assert rows(ws=NUL) == rows(wsb=8) == WORKSPACE


def test_move_refusals():
    for f in (gather, combine, combine_back):
        assert f(T=-1) == f(H=-8) == f(H=H + 4) == f(k=0) == f(k=65) == f(T=1 << 30) == SHAPE
    assert gather(xt=2) == combine(yt=2) == combine(ot=2) == combine_back(dt=2) == combine_back(yt=-1) == DTYPE
    assert gather(x=NUL) == gather(s=NUL) == gather(out=NUL) == combine(y=NUL) == combine(r=NUL) == combine(out=NUL) == NULL
    assert [combine_back(**{n: NUL}) for n in ("d", "y", "r", "w", "s", "dy", "dw")] == [NULL] * 7
    assert gather(x=P(0, 8)) == gather(s=P(1, 2)) == combine(w=P(2, 2)) == combine(out=P(3, 4)) == ALIGN
    assert combine_back(dw=P(6, 2)) == combine_back(dy=P(5, 8)) == combine_back(s=P(4, 1)) == ALIGN
    assert gather(ldx=H - 8) == gather(ldo=H + 4) == combine(ldy=H + 1) == combine_back(ldg=8) == combine_back(ldd=H + 2) == LD
    assert gather(out=P(0)) == gather(out=P(1)) == combine(out=P(0)) == combine(out=P(2)) == OVERLAP
    assert combine_back(dy=P(0)) == combine_back(dy=P(1)) == combine_back(dw=P(3)) == combine_back(dw=P(5)) == OVERLAP


def test_binding_refusals():
    x, e = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    w, n = torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32)
    y = torch.zeros(8, 16)
    for call in (lambda: fq.route_experts(x.half(), 2), lambda: fq.route_experts(x, 2, bias=torch.zeros(16).double()),
                 lambda: fq.route_experts_backward(w.double(), x, e), lambda: fq.route_experts_backward(w, x, e.long()),
                 lambda: fq.expert_rows(e.long(), 4), lambda: fq.gather_rows(x, n.long(), 2),
                 lambda: fq.combine_rows(y, e.long()), lambda: fq.combine_rows(y, e, w.double()),
                 lambda: fq.combine_rows_backward(x, y.half(), e, w, n)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fq.route_experts(x, 2), lambda: fq.route_experts(x, 2, score="max"),
                 lambda: fq.route_experts(x, 2, bias=torch.zeros(15)), lambda: fq.route_experts(x.t()[:, ::2], 2),
                 lambda: fq.route_experts_backward(w[:3], x, e), lambda: fq.route_experts_backward(w, x, e[:, :1]),
                 lambda: fq.expert_rows(e, 4), lambda: fq.expert_rows(e.t(), 4), lambda: fq.gather_rows(x, n, 3),
                 lambda: fq.gather_rows(x, n, 2), lambda: fq.combine_rows(y[:7], e), lambda: fq.combine_rows(y, e, w.t()),
                 lambda: fq.combine_rows_backward(x, y, e, w, n[:7])):
        with pytest.raises(ValueError):
            call()
