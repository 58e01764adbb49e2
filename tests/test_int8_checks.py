"""Refusals of the 8-bit integer entry points, without a GPU: the C ABI's statuses on fake pointers and the Python
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
P = lambda i, plus=0: ctypes.c_void_p(0x10000000 * (i + 1) + plus)
NUL = ctypes.c_void_p(0)
M, N, K, E = 300, 70, 160, 4
BIG = 1 << 40


def rows(x=P(0), xt=0, R=M, C=K, ldx=K, q=P(1), ldq=K, s=P(2)):
    return fq.lib().fp8bq_quantize_int8(x, xt, R, C, ldx, q, ldq, s, NUL)


def cols(x=P(0), xt=0, R=M, C=K, ldx=K, q=P(1), ldq=304, s=P(2), ws=P(3), wsb=BIG):
    return fq.lib().fp8bq_quantize_int8_t(x, xt, R, C, ldx, q, ldq, s, ws, wsb, NUL)


def gemm(M=M, N=N, K=K, a=P(0), lda=K, sa=P(1), b=P(2), ldb=K, sb=P(3), c=P(4), ct=0, ldc=N, ws=P(8), wsb=BIG,
         grouped=False, E=E, off=P(9)):
    if grouped:
        return fq.lib().fp8bq_grouped_gemm_int8(E, M, N, K, off, a, lda, sa, b, ldb, sb, c, ct, ldc, ws, wsb, NUL)
    return fq.lib().fp8bq_gemm_int8(M, N, K, a, lda, sa, b, ldb, sb, c, ct, ldc, ws, wsb, NUL)


def linear(M=M, N=N, K=K, x=P(0), xt=0, ldx=K, b=P(2), ldb=K, sb=P(3), c=P(4), ct=0, ldc=N, ws=P(8), wsb=BIG,
           grouped=False, E=E, off=P(9)):
    if grouped:
        return fq.lib().fp8bq_grouped_linear_int8(E, M, N, K, off, x, xt, ldx, b, ldb, sb, c, ct, ldc, ws, wsb, NUL)
    return fq.lib().fp8bq_linear_int8(M, N, K, x, xt, ldx, b, ldb, sb, c, ct, ldc, ws, wsb, NUL)


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bq_int8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp8bq_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 11
    for n in names:
        assert hasattr(fq, n) and hasattr(fq.lib(), n), n


@pytest.mark.skipif(HAVE_GPU, reason="fake pointers: checks the no-device path")
def test_valid_arguments_reach_the_device_check():
    assert rows() == cols() == DEVICE
    assert rows(xt=1) == cols(xt=1) == cols(C=8, ldx=8) == DEVICE
    for g in (False, True):
        assert gemm(grouped=g) == linear(grouped=g) == DEVICE
        assert gemm(grouped=g, ct=1, ldc=N + 1) == linear(grouped=g, xt=1) == DEVICE
    assert gemm(ct=2) == DEVICE
    assert gemm(K=(1 << 17) - 16, lda=1 << 17, ldb=1 << 17) == DEVICE


def test_empty_calls_succeed():
    assert rows(R=0) == rows(C=0) == cols(R=0) == cols(C=0) == OK
    for g in (False, True):
        assert gemm(M=0, grouped=g) == gemm(N=0, grouped=g) == linear(M=0, grouped=g) == linear(N=0, grouped=g) == OK


def test_quantizer_refusals():
    for f in (rows, cols):
        assert f(xt=2) == f(xt=-1) == DTYPE
        assert f(R=-1) == f(C=-16) == f(C=K + 4) == f(R=1 << 30) == f(C=1 << 30) == f(R=1 << 31) == SHAPE
        assert f(x=NUL) == f(q=NUL) == f(s=NUL) == NULL
        assert f(x=P(0, 8)) == f(q=P(1, 4)) == f(s=P(2, 4)) == ALIGN
        assert f(ldx=K - 8) == f(ldx=K + 1) == f(ldq=K - 16) == f(ldq=313) == LD
        assert f(q=P(0)) == f(s=P(0)) == f(s=P(1)) == OVERLAP
    assert rows(C=K - 8) == SHAPE
    assert cols(ldq=300) == cols(ldq=288) == LD
    assert cols(ws=NUL) == cols(wsb=16) == WORKSPACE
    assert cols(ws=P(3, 4)) == ALIGN and cols(ws=P(1)) == OVERLAP


@pytest.mark.parametrize("grouped", [False, True])
def test_product_refusals(grouped):
    def g(**k):
        return gemm(grouped=grouped, **k)

    def l(**k):
        return linear(grouped=grouped, **k)

    for f in (g, l):
        assert f(ct=3) == f(ct=-1) == DTYPE
        assert f(M=-1) == f(N=-1) == f(K=-16) == f(K=K + 8) == f(K=1 << 17) == f(M=1 << 30) == f(N=1 << 30) == SHAPE
        assert f(b=NUL) == f(sb=NUL) == f(c=NUL) == NULL
        assert f(b=P(2, 8)) == f(sb=P(3, 4)) == f(c=P(4, 2)) == ALIGN
        assert f(ldb=K - 16) == f(ldb=K + 8) == f(ldc=N - 1) == f(ldb=1 << 24) == LD
        assert f(c=P(2)) == f(c=P(3)) == OVERLAP
    assert g(a=NUL) == g(sa=NUL) == l(x=NUL) == NULL
    assert g(lda=1 << 24) == LD and g(c=P(0)) == g(c=P(1)) == l(c=P(0)) == OVERLAP
    assert l(xt=2) == DTYPE and l(ct=2) == DTYPE
    assert l(ws=NUL) == l(wsb=16) == WORKSPACE
    assert l(ws=P(8, 4)) == ALIGN and l(ws=P(4)) == OVERLAP
    if grouped:
        assert g(ct=2) == DTYPE and g(off=NUL) == NULL and g(off=P(9, 4)) == ALIGN
        assert g(E=0) == g(E=513) == l(E=0) == g(K=0, lda=16, ldb=16) == SHAPE
        assert g(c=P(9)) == OVERLAP


def test_workspace_sizes():
    lib = fq.lib()
    assert lib.fp8bq_linear_int8_workspace_size(1, 2048, 2048) == 0
    assert lib.fp8bq_linear_int8_workspace_size(1000, 2048, 2048) >= 1000 * 2048 + 4000
    assert lib.fp8bq_gemm_int8_workspace_size(64, 64, 20000) > 0
    for f in (lib.fp8bq_gemm_int8_workspace_size, lib.fp8bq_linear_int8_workspace_size):
        assert f(-1, 8, 16) == f(8, 8, 17) == f(8, 8, 1 << 17) == f(1 << 62, 1 << 62, 16) == 0
    assert lib.fp8bq_grouped_gemm_int8_workspace_size(0, 8, 8, 16) == lib.fp8bq_grouped_linear_int8_workspace_size(513, 8, 8, 16) == 0
    assert lib.fp8bq_quantize_int8_t_workspace_size(-1, 8) == lib.fp8bq_quantize_int8_t_workspace_size(8, 0) == 0
    assert lib.fp8bq_quantize_int8_t_workspace_size(1 << 62, 8) == 0


def test_binding_refusals():
    x = torch.zeros(4, 32)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    off = torch.tensor([0, 4])
    for call in (lambda: fq.fp8bq_quantize_int8(x.half(), q, s), lambda: fq.fp8bq_quantize_int8(x, q.view(torch.uint8), s),
                 lambda: fq.fp8bq_quantize_int8(x, q, s.double()), lambda: fq.gemm_int8(q, s, q, None),
                 lambda: fq.gemm_int8(q.view(torch.uint8), s, q, s), lambda: fq.linear_int8(q, q, s),
                 lambda: fq.grouped_linear_int8(x, None, q, s)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fq.quantize_int8(x), lambda: fq.gemm_int8(q, s, q, s), lambda: fq.linear_int8(x, q, s),
                 lambda: fq.grouped_linear_int8(x, off, q, s),  # (on the CPU)
                 lambda: fq.fp8bq_quantize_int8(x, q[:, :16], s), lambda: fq.fp8bq_quantize_int8(x, q, s[:3]),
                 lambda: fq.fp8bq_quantize_int8(x, q, torch.zeros(8)[::2]),
                 lambda: fq.fp8bq_quantize_int8(torch.zeros(32, 4).t(), q, s),
                 lambda: fq.gemm_int8(q, s, q[:, :16], s), lambda: fq.gemm_int8(q, s, q, s, accumulate=True),
                 lambda: fq.grouped_linear_int8(x, torch.tensor([0, 1, 2, 4]), q, s)):
        with pytest.raises(ValueError):
            call()
