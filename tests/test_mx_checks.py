"""Refusals of the MXFP4 entry points, without a GPU: the C ABI's statuses on fake pointers and the Python
binding's checks."""

import ctypes
import os
import re

import pytest
import torch

import fp8_blockwise_quantized_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, LD, ALIGN, DTYPE, FORMAT, WORKSPACE, DEVICE, LAUNCH, OVERLAP, VALUE = range(12)
HAVE_GPU = torch.cuda.is_available()
P = lambda i: ctypes.c_void_p(0x10000000 * (i + 1))
NUL = ctypes.c_void_p(0)
M, N, K, E = 300, 70, 160, 4
BIG = 1 << 40


def quant(x=P(0), xt=0, R=M, C=K, ldx=K, q=P(1), ldq=K // 2, s=P(2), lds=M, qt=P(3), ldqt=160, st=P(4), ldst=K):
    return fq.lib().fp8bq_quantize_mxfp4(x, xt, R, C, ldx, q, ldq, s, lds, qt, ldqt, st, ldst, NUL)


def gemm(M=M, N=N, K=K, a=P(0), lda=K // 2, sa=P(1), ldsa=M, b=P(2), ldb=K // 2, sb=P(3), ldsb=E * N, c=P(4), ct=0,
         ldc=N, ws=P(8), wsb=BIG, grouped=False, E=E, off=P(9)):
    if grouped:
        return fq.lib().fp8bq_grouped_gemm_mxfp4(E, M, N, K, off, a, lda, sa, ldsa, b, ldb, sb, ldsb, c, ct, ldc, ws, wsb,
                                                 NUL)
    return fq.lib().fp8bq_gemm_mxfp4(M, N, K, a, lda, sa, ldsa, b, ldb, sb, ldsb, c, ct, ldc, ws, wsb, NUL)


def linear(M=M, N=N, K=K, x=P(0), xt=0, ldx=K, b=P(2), ldb=K // 2, sb=P(3), ldsb=E * N, c=P(4), ct=0, ldc=N, ws=P(8),
           wsb=BIG, grouped=False, E=E, off=P(9)):
    if grouped:
        return fq.lib().fp8bq_grouped_linear_mxfp4(E, M, N, K, off, x, xt, ldx, b, ldb, sb, ldsb, c, ct, ldc, ws, wsb, NUL)
    return fq.lib().fp8bq_linear_mxfp4(M, N, K, x, xt, ldx, b, ldb, sb, ldsb, c, ct, ldc, ws, wsb, NUL)


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bq_mx.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp8bq_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 9
    for n in names:
        assert hasattr(fq, n) and hasattr(fq.lib(), n), n


@pytest.mark.skipif(HAVE_GPU, reason="fake pointers: checks the no-device path")
def test_valid_arguments_reach_the_device_check():
    assert quant() == DEVICE
    assert quant(q=NUL, s=NUL) == DEVICE and quant(qt=NUL, st=NUL) == DEVICE
    assert quant(C=40, ldx=40, q=NUL, s=NUL, ldst=40) == DEVICE
    for g in (False, True):
        assert gemm(grouped=g) == DEVICE and linear(grouped=g) == DEVICE
        assert gemm(grouped=g, ct=1, ldc=N + 1) == DEVICE and linear(grouped=g, xt=1) == DEVICE
    assert gemm(ct=2) == DEVICE


def test_empty_calls_succeed():
    assert quant(R=0) == OK and quant(C=0) == OK
    for g in (False, True):
        assert gemm(M=0, grouped=g) == OK and gemm(N=0, grouped=g) == OK and linear(M=0, grouped=g) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), DTYPE), (dict(R=-1), SHAPE), (dict(C=44), SHAPE), (dict(C=40), SHAPE), (dict(R=1 << 31), SHAPE),
    (dict(x=NUL), NULL), (dict(q=NUL), NULL), (dict(st=NUL), NULL), (dict(q=NUL, s=NUL, qt=NUL, st=NUL), NULL),
    (dict(x=ctypes.c_void_p(0x1008)), ALIGN), (dict(q=ctypes.c_void_p(0x1008)), ALIGN), (dict(ldq=K // 2 - 16), LD),
    (dict(ldq=K // 2 + 8), LD), (dict(ldqt=144), LD), (dict(lds=M - 1), LD), (dict(ldx=K + 4), LD),
    (dict(q=P(0)), OVERLAP), (dict(qt=P(1)), OVERLAP), (dict(st=P(2)), OVERLAP)])
def test_quantizer_refusals(kw, status):
    assert quant(**kw) == status


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(ct=3), DTYPE), (dict(ct=-1), DTYPE), (dict(M=-1), SHAPE), (dict(K=40), SHAPE), (dict(M=1 << 30), SHAPE),
    (dict(N=1 << 30), SHAPE), (dict(b=NUL), NULL), (dict(sb=NUL), NULL), (dict(c=NUL), NULL),
    (dict(b=ctypes.c_void_p(0x1008)), ALIGN), (dict(ldb=K // 2 - 16), LD), (dict(ldb=K // 2 + 8), LD),
    (dict(ldsb=N - 1), LD), (dict(ldc=N - 1), LD), (dict(c=P(2)), OVERLAP), (dict(c=P(3)), OVERLAP),
    (dict(ldb=1 << 25), LD)])
def test_product_refusals(grouped, kw, status):
    assert gemm(grouped=grouped, **kw) == status
    assert linear(grouped=grouped, **kw) == status


@pytest.mark.parametrize("grouped", [False, True])
def test_product_refusals_of_one_kind(grouped):
    assert gemm(a=NUL, grouped=grouped) == NULL and gemm(sa=NUL, grouped=grouped) == NULL
    assert gemm(lda=K // 2 + 8, grouped=grouped) == LD and gemm(ldsa=M - 1, grouped=grouped) == LD
    assert gemm(c=P(1), grouped=grouped) == OVERLAP
    assert linear(x=NUL, grouped=grouped) == NULL and linear(ldx=K + 4, grouped=grouped) == LD
    assert linear(xt=2, grouped=grouped) == DTYPE and linear(c=P(0), grouped=grouped) == OVERLAP
    assert linear(ws=NUL, wsb=0, grouped=grouped) == WORKSPACE  # 300 tokens: x's codes need space
    assert linear(ws=P(2), grouped=grouped) == OVERLAP and linear(ws=ctypes.c_void_p(0x1008), grouped=grouped) == ALIGN


def test_grouped_refusals():
    for call in (gemm, linear):
        assert call(grouped=True, E=0) == SHAPE and call(grouped=True, E=513) == SHAPE
        assert call(grouped=True, off=NUL) == NULL and call(grouped=True, off=ctypes.c_void_p(0x1004)) == ALIGN
        assert call(grouped=True, K=0) == SHAPE and call(grouped=True, c=P(9)) == OVERLAP


def test_workspace_sizes():
    assert fq.fp8bq_linear_mxfp4_workspace_size(1, 2048, 2048) == 0
    assert fq.fp8bq_linear_mxfp4_workspace_size(4096, 2048, 2048) >= 4096 * 1024 + 4096 * 64
    assert fq.fp8bq_linear_mxfp4_workspace_size(-1, 2048, 2048) == 0
    assert fq.fp8bq_linear_mxfp4_workspace_size(64, 64, 33) == 0
    assert fq.fp8bq_linear_mxfp4_workspace_size(4, 64, 0) == 0 and fq.fp8bq_gemm_mxfp4_workspace_size(4, 64, 0) == 0
    assert fq.fp8bq_grouped_linear_mxfp4_workspace_size(0, 64, 64, 64) == 0
    assert fq.fp8bq_grouped_linear_mxfp4_workspace_size(64, 6, 2816, 2048) == 0


def t(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_mismatched_tensors():
    a = dict(qa=t(M, K // 2), sa=t(2, M, 4), qb=t(N, K // 2), sb=t(2, N, 4), c=t(M, N, dtype=torch.bfloat16))
    for kw, exc in ((dict(sa=t(1, M, 4)), ValueError), (dict(sa=t(2, M, 4, dtype=torch.int8)), TypeError),
                    (dict(qb=t(N, K)), ValueError), (dict(c=t(M, N + 1, dtype=torch.bfloat16)), ValueError),
                    (dict(c=t(M, N, dtype=torch.float16)), TypeError), (dict(), ValueError)):  # (the last: host tensors)
        v = {**a, **kw}
        with pytest.raises(exc):
            fq.fp8bq_gemm_mxfp4(v["qa"], v["sa"], v["qb"], v["sb"], v["c"])
    with pytest.raises(TypeError):
        fq.fp8bq_gemm_mxfp4(a["qa"], a["sa"], a["qb"], a["sb"], a["c"], accumulate=True)
    with pytest.raises(ValueError):
        fq.gemm_mxfp4(a["qa"], a["sa"], a["qb"], a["sb"], accumulate=True)
    with pytest.raises(ValueError):
        fq.fp8bq_quantize_mxfp4(t(M, K, dtype=torch.bfloat16), t(M, K // 2), t(2, M, 3), None, None)
