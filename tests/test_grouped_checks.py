"""Refusals of the grouped entry points, without a GPU: the C ABI's statuses on fake pointers, the Python
binding's checks, and the padded row count."""

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
E, T, N, K = 4, 300, 256, 384
TP = 768


def quant(x=P(0), xt=0, T=T, C=K, ldx=K, off=P(9), E=E, fr=0, q=P(1), ldq=K, s=P(2), lds=304, fc=0, qt=P(3), ldqt=TP,
          st=P(4), ldst=K, padded=TP):
    return fq.lib().fp8bq_quantize_act_grouped(x, xt, T, C, ldx, off, E, fr, q, ldq, s, lds, fc, qt, ldqt, st, ldst,
                                               padded, NUL)


def gemm(op="fprop", E=E, T=T, N=N, K=K, off=P(9), a=P(0), lda=None, sa=P(1), ldsa=None, fa=0, b=P(2), ldb=None,
         sb=P(3), ldsb=None, fb=0, out=P(4), ot=0, ldo=None, ws=NUL, ws_bytes=0):
    if op == "wgrad":
        T = TP if T == 300 else T
    d = {"fprop": (K, 304, K, 3, N), "dgrad": (N, 304, E * N, 3, K), "wgrad": (T, N, T, K, K)}[op]
    lda, ldsa, ldb, ldsb, ldo = (v if v is not None else w for v, w in zip((lda, ldsa, ldb, ldsb, ldo), d))
    space = (ws, ws_bytes) if op == "wgrad" else ()
    return getattr(fq.lib(), "fp8bq_grouped_gemm_" + op)(E, T, N, K, off, a, lda, sa, ldsa, fa, b, ldb, sb, ldsb, fb,
                                                         out, ot, ldo, *space, NUL)


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bq_grouped.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp8bq_[a-z0-9_]+)\s*\(", text))
    assert names == {"fp8bq_grouped_padded_rows", "fp8bq_quantize_act_grouped", "fp8bq_grouped_gemm_fprop",
                     "fp8bq_grouped_gemm_dgrad", "fp8bq_grouped_gemm_wgrad",
                     "fp8bq_grouped_gemm_wgrad_workspace_size"}
    for n in names:
        assert hasattr(fq, n) and hasattr(fq.lib(), n)


@pytest.mark.skipif(HAVE_GPU, reason="fake pointers: checks the no-device path")
def test_valid_arguments_reach_the_device_check():
    assert quant() == DEVICE
    assert quant(q=NUL, s=NUL) == DEVICE
    for op in ("fprop", "dgrad", "wgrad"):
        assert gemm(op) == DEVICE, op
    assert gemm("wgrad", ot=2) == DEVICE


def test_empty_calls_succeed():
    assert quant(T=0, padded=0) == OK
    assert gemm("fprop", T=0) == OK and gemm("dgrad", T=0) == OK
    assert gemm("fprop", N=0) == OK and gemm("wgrad", K=0) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), DTYPE), (dict(fc=2), FORMAT), (dict(fr=3), FORMAT), (dict(E=0), SHAPE), (dict(E=513), SHAPE),
    (dict(T=-1), SHAPE), (dict(C=100), SHAPE), (dict(padded=640), SHAPE), (dict(padded=TP + 64), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(off=NUL), NULL), (dict(off=ctypes.c_void_p(0x1004)), ALIGN), (dict(qt=NUL), NULL),
    (dict(q=NUL), NULL), (dict(s=NUL), NULL), (dict(ldqt=TP - 16), LD), (dict(ldx=K - 8), LD), (dict(lds=301), LD),
    (dict(qt=P(0)), OVERLAP), (dict(q=P(3)), OVERLAP), (dict(st=P(9)), OVERLAP)])
def test_quantizer_refusals(kw, status):
    assert quant(**kw) == status


@pytest.mark.parametrize("op", ["fprop", "dgrad", "wgrad"])
@pytest.mark.parametrize("kw,status", [
    (dict(fa=2), FORMAT), (dict(fb=-1), FORMAT), (dict(ot=3), DTYPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE),
    (dict(N=100), SHAPE), (dict(K=100), SHAPE), (dict(N=1 << 29), SHAPE), (dict(off=NUL), NULL),
    (dict(off=ctypes.c_void_p(0x1004)), ALIGN), (dict(a=NUL), NULL), (dict(out=NUL), NULL),
    (dict(a=ctypes.c_void_p(0x1008)), ALIGN), (dict(ldb=128), LD), (dict(ldo=128), LD), (dict(out=P(0)), OVERLAP),
    (dict(out=P(9)), OVERLAP), (dict(lda=1 << 25), LD)])
def test_product_refusals(op, kw, status):
    assert gemm(op, **kw) == status


def test_product_refusals_of_one_op():
    assert gemm("fprop", ot=2) == DTYPE and gemm("dgrad", ot=2) == DTYPE
    assert gemm("wgrad", T=700) == SHAPE
    assert gemm("fprop", K=0) == SHAPE and gemm("dgrad", N=0) == SHAPE


def test_weight_gradient_workspace():
    """Needed only to split long experts: absent for few tokens, refused when too small, misaligned or shared."""
    size = fq.fp8bq_grouped_gemm_wgrad_workspace_size
    assert size(4, 768, 256, 384) == 0 and size(4, 0, 256, 384) == 0
    for bad in ((0, 8192, 128, 128), (513, 8192, 128, 128), (4, 8200, 128, 128), (4, 8192, 100, 128), (4, -128, 128, 128)):
        assert size(*bad) == 0
    n = size(4, 8192, 128, 256)
    assert n > 0 and (n - 256) % (128 * 256 * 4) == 0
    if HAVE_GPU:
        return  # (fake pointers)
    big = dict(E=4, T=8192, N=128, K=256)
    assert gemm("wgrad", **big) == DEVICE and gemm("wgrad", ws=P(5), ws_bytes=n, **big) == DEVICE


def test_padded_rows_hold_any_shares():
    for T_, E_ in ((1, 1), (7, 3), (127, 1), (128, 1), (129, 1), (300, 2), (600, 4)):
        p = fq.fp8bq_grouped_padded_rows(T_, E_)
        used = min(T_, E_)
        # the most blocks: every expert but one has one token past a whole number of blocks
        most, spare = used, T_ - used
        most += spare // 128
        assert p % 128 == 0 and 128 * most <= p <= T_ + 127 * used
    assert fq.fp8bq_grouped_padded_rows(0, 5) == 0
    assert fq.fp8bq_grouped_padded_rows(-1, 3) == 0 and fq.fp8bq_grouped_padded_rows(5, 513) == 0


def t(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_mismatched_tensors():
    off = t(E + 1, dtype=torch.int64)
    f32, bf = torch.float32, torch.bfloat16
    a = dict(qx=t(T, K), sx=t(K // 128, T, dtype=f32), off=off, qw=t(E * N, K), sw=t(E * N // 128, K // 128, dtype=f32),
             y=t(T, N, dtype=bf))

    def call(**kw):
        v = {**a, **kw}
        fq.fp8bq_grouped_gemm_fprop(v["qx"], v["sx"], fq.E4M3, v["off"], v["qw"], v["sw"], fq.E4M3, v["y"])

    for kw, exc in ((dict(off=off.int()), TypeError), (dict(off=off[:1]), ValueError), (dict(off=off[None]), ValueError),
                    (dict(qw=t(E * N + 1, K)), ValueError), (dict(sw=t(E, K // 128, dtype=f32)), ValueError),
                    (dict(y=t(T, N, dtype=torch.float16)), TypeError), (dict(y=t(T - 1, N, dtype=bf)), ValueError),
                    (dict(off=t(2 * (E + 1), dtype=torch.int64)[::2]), ValueError), (dict(), ValueError)):
        with pytest.raises(exc):  # (the last: host tensors)
            call(**kw)
