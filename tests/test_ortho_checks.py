"""Refusals of the orthogonalization, without a GPU: the C ABI's statuses on fake pointers and the Python binding's checks."""

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
B, R, C = 3, 50, 70
BIG = 1 << 40
MUON = (3.4445, -4.7750, 2.0315)


def ortho(g=P(0), gt=0, B=B, R=R, C=C, ldg=C, gs=R * C, steps=2, coef=MUON * 2, eps=1e-7, out=P(1), ldo=C, os_=R * C, ws=P(2),
          wsb=BIG):
    c = (ctypes.c_double * len(coef))(*coef) if coef is not None else NUL
    return fq.lib().fp8bq_orthogonalize(g, gt, B, R, C, ldg, gs, steps, c, eps, out, ldo, os_, ws, wsb, NUL)


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bq_ortho.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp8bq_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 2
    for n in names:
        assert hasattr(fq, n) and hasattr(fq.lib(), n), n


@pytest.mark.skipif(HAVE_GPU, reason="fake pointers: checks the no-device path")
def test_valid_arguments_reach_the_device_check():
    assert ortho() == ortho(gt=1) == ortho(g=P(0, 2), out=P(1, 6)) == ortho(ldg=C + 1, gs=R * (C + 1)) == DEVICE
    assert ortho(B=1, gs=0, os_=0) == DEVICE


def test_empty_calls_succeed():
    assert ortho(B=0) == ortho(R=0) == ortho(C=0) == OK


def test_refusals():
    assert ortho(gt=2) == DTYPE
    assert ortho(B=-1) == ortho(R=-1) == ortho(C=-1) == ortho(B=4097) == ortho(R=(1 << 20) + 1) == ortho(C=(1 << 20) + 1, ldg=1 << 21,
                                                                                                 ldo=1 << 21) == SHAPE
    assert ortho(B=4096, R=1 << 20, C=1 << 20, ldg=1 << 20, ldo=1 << 20, gs=1 << 40, os_=1 << 40) == SHAPE
    assert ortho(steps=0) == ortho(steps=65, coef=MUON * 65) == ortho(eps=0.0) == ortho(eps=-1.0) == VALUE
    assert ortho(eps=float("nan")) == ortho(eps=float("inf")) == ortho(coef=(1.0, 2.0, float("nan")) * 2) == VALUE
    assert ortho(g=NUL) == ortho(out=NUL) == ortho(coef=None) == NULL
    assert ortho(ldg=C - 1) == ortho(ldo=C - 1) == ortho(gs=R * C - 1) == ortho(os_=R * C - 1) == LD
    assert ortho(g=P(0, 1)) == ortho(gt=1, g=P(0, 2)) == ortho(out=P(1, 1)) == ortho(ws=P(2, 8)) == ALIGN
    assert ortho(out=P(0)) == ortho(ws=P(0)) == ortho(ws=P(1)) == OVERLAP
    assert ortho(ws=NUL) == ortho(wsb=100) == WORKSPACE


def test_workspace_sizes():
    size = fq.lib().fp8bq_orthogonalize_workspace_size
    assert size(1, 2048, 2048) >= 12 * 2048 * 2048
    assert size(0, 4, 4) == size(1, -1, 4) == size(1, 4, 1 << 21) == size(4096, 1 << 20, 1 << 20) == 0


def test_binding_refusals():
    g = torch.zeros(8, 16)
    for call in (lambda: fq.orthogonalize(g.half()), lambda: fq.orthogonalize(g, out=g)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fq.orthogonalize(g), lambda: fq.orthogonalize(g[0]), lambda: fq.orthogonalize(g, coefficients=[MUON]),
                 lambda: fq.orthogonalize(g, coefficients=[(1.0, 2.0)] * 5), lambda: fq.orthogonalize(g.t()),
                 lambda: fq.orthogonalize(g, out=g[:4].bfloat16())):
        with pytest.raises(ValueError):
            call()
