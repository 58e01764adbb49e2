"""The products on the planner's larger tiles (tile_cases.py; test_planned_tiles.py holds the sizes to those tiles): every
output type, edges that end inside a tile, guards around outputs and workspaces.  Compared on the device with the
float64 product of the same codes: within 1e-4 ||a|| ||b|| (the FP32 rule of parity.py), and a BF16 output half a unit
in its last place more, 2^-8 |y|."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import synth
from parity import F32_ABS, say
from test_gpu_grouped_split import expected, operands
from tile_cases import MX_GROUPED, MX_SPLIT, ROWS, WGRAD

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def guarded(rows, cols, dtype, ld=None):
    """A buffer of sevens and the matrix inside it."""
    big = torch.full((rows + 12, ld or cols + 16), 7.0, dtype=dtype, device="cuda")
    return big, big[8:rows + 8, :cols]


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


def offsets(counts, before=0):
    return torch.from_numpy(before + np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)).cuda()


def bound(a, b):
    """The float64 product a . b^T and the FP32 bound around it."""
    return a @ b.t().contiguous(), F32_ABS * torch.outer(a.norm(dim=1), b.norm(dim=1))


def decoded(q, s):
    """float64 values of E4M3 codes [R, C] with scales [C / 128, R]."""
    return q.view(torch.float8_e4m3fn).double() * s.double().t().repeat_interleave(128, 1)


@pytest.mark.parametrize("name", sorted(ROWS))
def test_grouped_rows(name):
    say("tiles rows", name)
    counts, N, K, _, _ = ROWS[name]
    E, T = len(counts), sum(counts)
    off = offsets(counts)
    x = synth.random_bf16((T, K), 700, 1.0, outliers=True).cuda()
    dy = synth.random_bf16((T, N), 701, 1e-3).cuda()
    w = synth.random_bf16((E * N, K), 702, 0.02).cuda()
    qw, sw, qwt = fq.quantize_weight_dual(w, fq.E4M3)
    (qx, sx), (qd, sd) = fq.quantize_act_1x128(x), fq.quantize_act_1x128(dy)
    outs = []
    for dtype in DTYPES:
        by, y = guarded(T, N, dtype)
        bd, dx = guarded(T, K, dtype)
        fq.grouped_gemm_fprop(qx, sx, off, qw, sw, out=y)
        fq.grouped_gemm_dgrad(qd, sd, off, qwt, sw, out=dx)
        outs.append((by, y, bd, dx))
    wd = qw.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    xd, dd = decoded(qx, sx), decoded(qd, sd)
    p = 0
    for e, n in enumerate(counts):
        rows, we = slice(p, p + n), wd[e * N:(e + 1) * N]
        p += n
        wanty, wantd = bound(xd[rows], we), bound(dd[rows], we.t())
        for _, y, _, dx in outs:
            assert close(y[rows], *wanty), ("fprop", e, y.dtype)
            assert close(dx[rows], *wantd), ("dgrad", e, dx.dtype)
    for by, y, bd, dx in outs:
        assert untouched(by, y) and untouched(bd, dx)


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mx_decoded(q, s):
    """float64 values of packed codes [R, K / 2] with scale words [ceil(K / 128), R, 4]."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=q.device)
    R, K = q.shape[0], 2 * q.shape[1]
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).view(R, K // 32, 32)
    b = s.transpose(0, 1).reshape(R, -1)[:, :K // 32].double()
    return (v * torch.exp2(b - 127).unsqueeze(-1)).view(R, K)


@pytest.mark.parametrize("name", sorted(MX_GROUPED))
def test_grouped_mxfp4(name):
    say("tiles mx grouped", name)
    counts, N, K, _ = MX_GROUPED[name]
    E, before, after = len(counts), 3, 70
    T = before + sum(counts) + after
    off = offsets(counts, before)
    x = synth.random_bf16((T, K), 710, 1.0, outliers=True).cuda()
    qw, sw = fq.quantize_mxfp4(synth.random_bf16((E * N, K), 711, 0.02).cuda())
    qx, sx = fq.quantize_mxfp4(x)
    outs = []
    for dtype in DTYPES:
        outs.append(guarded(T, N, dtype))
        fq.grouped_gemm_mxfp4(qx, sx, off, qw, sw, out=outs[-1][1])
        outs.append(guarded(T, N, dtype))
        fq.grouped_linear_mxfp4(x, off, qw, sw, out=outs[-1][1])
    xd, wd = mx_decoded(qx, sx), mx_decoded(qw, sw)
    p = before
    for e, n in enumerate(counts):
        want = bound(xd[p:p + n], wd[e * N:(e + 1) * N])
        for _, y in outs:
            assert close(y[p:p + n], *want), (e, y.dtype)
        p += n
    for big, y in outs:
        y[before:T - after] = 7.0
        assert torch.all(big == 7.0)


@pytest.mark.parametrize("M,N,K,rows,parts", MX_SPLIT)
def test_split_mxfp4(M, N, K, rows, parts):
    say("tiles mx split", M, N, K)
    x = synth.random_bf16((M, K), 720, 1.0, outliers=True).cuda()
    qw, sw = fq.quantize_mxfp4(synth.random_bf16((N, K), 721, 0.02).cuda())
    qx, sx = fq.quantize_mxfp4(x)
    want = bound(mx_decoded(qx, sx), mx_decoded(qw, sw))
    spaces = []
    for size in (fq.fp8bq_gemm_mxfp4_workspace_size(M, N, K), fq.fp8bq_linear_mxfp4_workspace_size(M, N, K)):
        assert size >= 4 * parts * M * N
        spaces.append((size, torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")))  # (NaNs, and a guard)
    (n, ws), (nl, wl) = spaces
    for dtype in DTYPES:
        for call in (lambda out: fq.gemm_mxfp4(qx, sx, qw, sw, out=out, ws=ws[:n]),
                     lambda out: fq.linear_mxfp4(x, qw, sw, out=out, ws=wl[:nl])):
            big, y = guarded(M, N, dtype)
            call(y)
            assert close(y, *want)
            assert untouched(big, y)
    one = fq.gemm_mxfp4(qx, sx, qw, sw, out_dtype=torch.float32)
    start = torch.randn(M, N, device="cuda")
    big, acc = guarded(M, N, torch.float32)
    acc.copy_(start)
    fq.gemm_mxfp4(qx, sx, qw, sw, out=acc, ws=ws[:n], accumulate=True)
    assert torch.equal(acc, start + one) and untouched(big, acc)
    assert torch.all(ws[n:] == 0xFF) and torch.all(wl[nl:] == 0xFF)


@pytest.mark.parametrize("M", [300, 1100])
def test_split_mxfp4_nan_blocks_reach_their_rows_only(M):
    say("tiles mx split nan", M)
    N, K = 1000, 11296
    x = synth.random_bf16((M, K), 730, 1.0)
    x[7, K - 5], x[M - 1, 3] = float("nan"), -float("inf")
    qw, sw = fq.quantize_mxfp4(synth.random_bf16((N, K), 731, 0.02).cuda())
    y = fq.linear_mxfp4(x.cuda(), qw, sw)
    rows = torch.isnan(y).any(1)
    assert torch.equal(rows, torch.isnan(y).all(1)) and rows.nonzero().flatten().tolist() == [7, M - 1]


# Outputs of 50 MB (BF16, rows of 8 KB; MXFP4 16 KB) and 100 MB (FP32) stay in the caches, parts of them go past: the two kinds of store
# give the same bits, and neither writes outside.

def codes(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 255, (rows, cols), dtype=torch.uint8, device="cuda", generator=g)


def finite_fp8(rows, cols, seed):
    q = codes(rows, cols, seed)
    return torch.where(q & 127 == 127, torch.zeros_like(q), q)  # (no E4M3 NaN)


def scales(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(rows, cols, device="cuda", generator=g) + 0.5


@pytest.mark.parametrize("dtype", DTYPES)
def test_kept_and_streamed_outputs_of_the_dense_products(dtype):
    say("tiles stores dense", dtype)
    M, N, K = 6500, 3968, 256
    q, s, w, sw = finite_fp8(M, K, 1), scales(K // 128, M, 2), finite_fp8(N, K, 3), scales(N // 128, K // 128, 4)
    big, y = guarded(M, N, dtype, 4096)
    fq.gemm_fprop(q, s, w, sw, out=y)
    half = M // 8 * 4
    for a, b in ((0, half), (half, M)):
        assert torch.equal(y[a:b], fq.gemm_fprop(q[a:b], s[:, a:b].contiguous(), w, sw, out_dtype=dtype))
    assert untouched(big, y)
    T, N, K = 256, 6400, 3968
    q, s, w, sw = finite_fp8(N, T, 5), scales(T // 128, N, 6), finite_fp8(K, T, 7), scales(T // 128, K, 8)
    big, y = guarded(N, K, dtype, 4096)
    fq.gemm_wgrad(q, s, w, sw, out=y)
    for a, b in ((0, 3200), (3200, N)):
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
    E, N, K = 4, 3968, 256
    T = 6500
    cuts = torch.tensor([0, 3, T // 3, T // 3, T], device="cuda")
    x, dy = (torch.randn(T, c, device="cuda").to(torch.bfloat16) for c in (K, N))
    w = torch.randn(E * N, K, device="cuda").to(torch.bfloat16)
    qw, sw, qwt = fq.quantize_weight_dual(w, fq.E4M3)
    q, s = fq.quantize_act_1x128(x)
    big, y = guarded(T, N, dtype, 4096)
    fq.grouped_gemm_fprop(q, s, cuts, qw, sw, out=y)
    for a, b, e in ((0, 3, 0), (3, T // 3, 1), (T // 3, T, 3)):
        one = fq.grouped_gemm_fprop(q[a:b], fq.quantize_act_1x128(x[a:b])[1], torch.tensor([0, b - a], device="cuda"),
                                    qw[e * N:(e + 1) * N], sw[e * N // 128:(e + 1) * N // 128].clone(), out_dtype=dtype)
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
    M, N, K = 6500, 3976, 320
    ld = 8192 if dtype == torch.bfloat16 else 4096
    x, w = (torch.randn(r, K, device="cuda").to(torch.bfloat16) for r in (M, N))
    qa, sa = fq.quantize_mxfp4(x)
    qb, sb = fq.quantize_mxfp4(w)
    big, y = guarded(M, N, dtype, ld)
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
    both, g = guarded(M, N, dtype, ld)
    fq.grouped_gemm_mxfp4(qa, sa, off, qe, se, out=g)
    assert torch.equal(g, y)
    assert untouched(big, y) and untouched(both, g)
