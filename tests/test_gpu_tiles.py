"""The products on the planner's larger tiles (tile_cases.py; test_planned_tiles.py holds the sizes to those tiles): every
output type, edges that end inside a tile, guards around outputs and workspaces.  Compared on the device with the
float64 product of the same codes: within 1e-4 ||a|| ||b|| (the FP32 rule of parity.py), and a BF16 output half a unit
in its last place more, 2^-8 |y|."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say
from test_gpu_grouped_split import expected, operands
from tile_cases import WGRAD

pytestmark = pytest.mark.gpu


def guarded(rows, cols, dtype):
    """A buffer of sevens and the matrix inside it."""
    big = torch.full((rows + 8, cols + 16), 7.0, dtype=dtype, device="cuda")
    return big, big[4:rows + 4, :cols]


def close(got, y, lim):
    if got.dtype == torch.bfloat16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
    return bool(torch.all((got.double() - y).abs() <= lim))


def untouched(big, inner):
    inner.fill_(7.0)
    return bool(torch.all(big == 7.0))


@pytest.mark.parametrize("name", sorted(WGRAD))
def test_grouped_weight_gradients(name):
    say("tiles wgrad", name)
    counts, N, K, _, split = WGRAD[name]
    E = len(counts)
    off, (qdyt, sdyt), (qxt, sxt) = operands(counts, N, K, 500)
    y, lim = expected(counts, qdyt, sdyt, qxt, sxt)
    size = fq.fp8bq_grouped_gemm_wgrad_workspace_size(E, qdyt.shape[1], N, K)
    assert (size > 0) == split
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(dw, space, **kw):
        fq.fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fq.E5M2, qxt, sxt, fq.E4M3, off, dw, ws=space, **kw)

    for space in (ws[:size], None) if split else (None,):
        big, one = guarded(E * N, K, torch.float32)
        run(one, space)
        assert close(one, y, lim)
        start = torch.randn(E * N, K, device="cuda")
        wide, acc = guarded(E * N, K, torch.float32)
        acc.copy_(start)
        run(acc, space, accumulate=True)
        assert torch.equal(acc, start + one)  # one FP32 addition an element
        half, dw = guarded(E * N, K, torch.bfloat16)
        run(dw, space)
        assert close(dw, y, lim)
        assert untouched(big, one) and untouched(wide, acc) and untouched(half, dw)
    assert torch.all(ws[size:] == 0xFF)


# Outputs of 105 to 120 MB stay in the caches, parts of them go past: the two kinds of store give the same bits, and neither
# writes outside.

def codes(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 255, (rows, cols), dtype=torch.uint8, device="cuda", generator=g)


def finite_fp8(rows, cols, seed):
    q = codes(rows, cols, seed)
    return torch.where(q & 127 == 127, torch.zeros_like(q), q)  # (no E4M3 NaN)


def scales(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(rows, cols, device="cuda", generator=g) + 0.5


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
def test_kept_and_streamed_outputs_of_the_dense_products(dtype):
    say("tiles stores dense", dtype)
    M, N, K = 26000 if dtype == torch.bfloat16 else 13000, 2048, 256
    q, s, w, sw = finite_fp8(M, K, 1), scales(K // 128, M, 2), finite_fp8(N, K, 3), scales(N // 128, K // 128, 4)
    big, y = guarded(M, N, dtype)
    fq.gemm_fprop(q, s, w, sw, out=y)
    half = M // 8 * 4
    for a, b in ((0, half), (half, M)):
        assert torch.equal(y[a:b], fq.gemm_fprop(q[a:b], s[:, a:b].contiguous(), w, sw, out_dtype=dtype))
    assert untouched(big, y)
    T, N, K = 256, 12800, 4096 if dtype == torch.bfloat16 else 2048
    q, s, w, sw = finite_fp8(N, T, 5), scales(T // 128, N, 6), finite_fp8(K, T, 7), scales(T // 128, K, 8)
    big, y = guarded(N, K, dtype)
    fq.gemm_wgrad(q, s, w, sw, out=y)
    for a, b in ((0, 6400), (6400, N)):
        assert torch.equal(y[a:b], fq.gemm_wgrad(q[a:b], s[:, a:b].contiguous(), w, sw, out_dtype=dtype))
    if dtype == torch.float32:
        start = torch.randn(N, K, device="cuda")
        acc = start.clone()
        fq.gemm_wgrad(q, s, w, sw, out=acc, accumulate=True)
        assert torch.equal(acc, start + y)
    assert untouched(big, y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_kept_and_streamed_outputs_of_the_grouped_products(dtype):
    say("tiles stores grouped", dtype)
    E, N, K = 4, 2048, 256
    T = 26000 if dtype == torch.bfloat16 else 13000
    cuts = torch.tensor([0, 3, T // 3, T // 3, T], device="cuda")
    x, dy = (torch.randn(T, c, device="cuda").to(torch.bfloat16) for c in (K, N))
    w = torch.randn(E * N, K, device="cuda").to(torch.bfloat16)
    qw, sw, qwt = fq.quantize_weight_dual(w, fq.E4M3)
    q, s = fq.quantize_act_1x128(x)
    big, y = guarded(T, N, dtype)
    fq.grouped_gemm_fprop(q, s, cuts, qw, sw, out=y)
    for a, b, e in ((0, 3, 0), (3, T // 3, 1), (T // 3, T, 3)):
        one = fq.grouped_gemm_fprop(q[a:b], fq.quantize_act_1x128(x[a:b])[1], torch.tensor([0, b - a], device="cuda"),
                                    qw[e * N:(e + 1) * N], sw[e * N // 128:(e + 1) * N // 128], out_dtype=dtype)
        assert torch.equal(y[a:b], one)
    assert untouched(big, y)
    E, N, K = 32, 1024, 1664 if dtype == torch.bfloat16 else 896
    counts = [70 * (e % 3) for e in range(E)]
    off, (qdyt, sdyt), (qxt, sxt) = operands(counts, N, K, 600)
    big, y = guarded(E * N, K, dtype)
    fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, off, fq.E5M2, out=y)
    want, lim = expected(counts, qdyt, sdyt, qxt, sxt)
    assert close(y, want, lim)
    assert untouched(big, y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_kept_and_streamed_outputs_of_the_mxfp4_products(dtype):
    say("tiles stores mx", dtype)
    M, N, K = 26000 if dtype == torch.bfloat16 else 13000, 2056, 320
    x, w = (torch.randn(r, K, device="cuda").to(torch.bfloat16) for r in (M, N))
    qa, sa = fq.quantize_mxfp4(x)
    qb, sb = fq.quantize_mxfp4(w)
    big, y = guarded(M, N, dtype)
    fq.gemm_mxfp4(qa, sa, qb, sb, out=y)
    half = M // 8 * 4
    for a, b in ((0, half), (half, M)):
        assert torch.equal(y[a:b], fq.gemm_mxfp4(qa[a:b], sa[:, a:b].contiguous(), qb, sb, out_dtype=dtype))
    if dtype == torch.float32:
        start = torch.randn(M, N, device="cuda")
        acc = start.clone()
        fq.gemm_mxfp4(qa, sa, qb, sb, out=acc, accumulate=True)
        assert torch.equal(acc, start + y)
    off = torch.tensor([0, 5, 5, M], device="cuda")
    qe, se = fq.quantize_mxfp4(torch.cat([w, w, w]))
    both, g = guarded(M, N, dtype)
    fq.grouped_gemm_mxfp4(qa, sa, off, qe, se, out=g)
    assert torch.equal(g, y)
    assert untouched(big, y) and untouched(both, g)
