"""8-bit integer quantizers and products against float64.

Codes and scales bit for bit.  A product's integer sum is exact; making it FP32 and multiplying by two scales rounds three
times, each by at most 2^-24 relative, and a BF16 output once more, by at most 2^-8."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def normal(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def codes(shape, seed, low=-127):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, 128, shape, generator=g, dtype=torch.int8)


def scales(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(n, generator=g) * 0.05 + 1e-4


def rule(x):
    """Codes and scales of x's rows on the CPU (IEEE divisions)."""
    v = x.float()
    s = torch.maximum(v.abs().amax(1) / torch.full((), 127.0), torch.full((), 1e-12))
    return torch.round(v / s.unsqueeze(1)).to(torch.int8), s


def exact(qa, sa, qb, sb):
    y = qa.cuda().double() @ qb.cuda().double().t()
    return y * sa.cuda().double().unsqueeze(1) * sb.cuda().double()


def limit(y, dtype):
    return y.abs() * (2.0 ** -8 if dtype == BF16 else 0.0) + y.abs() * 3.01 * 2.0 ** -24


def close(got, want, extra=0.0):
    torch.cuda.synchronize()
    off = (got.double() - want).abs()
    assert bool((off <= limit(want, got.dtype) + extra).all()), float((off - limit(want, got.dtype)).max())


def special(R, C, seed):
    """Ties, zeros, subnormals, the largest and the smallest values, a row of zeros."""
    x = normal((R, C), seed)
    g = torch.Generator().manual_seed(seed + 1)
    pick = torch.tensor([0.0, -0.0, 1e-40, -3e-45, 0.5, 1.5, -2.5, 63.5, 126.5, 127.0, -127.0, 3e38, -3e38, 2.0 ** -126])
    where = torch.rand(R, C, generator=g) < 0.3
    x[where] = pick[torch.randint(0, len(pick), (R, C), generator=g)][where]
    x[0] = 127.0 * torch.sign(normal((C,), seed + 2))
    x[0, :C // 2] = (torch.arange(C // 2) % 253 - 126) + 0.5  # scale 1: every value a tie
    if R > 2:
        x[1] = 0.0
        x[2] = x[2].clamp(-1e-38, 1e-38)
    return x


@pytest.mark.parametrize("R,C", [(1, 16), (3, 48), (17, 2048), (130, 4112), (64, 6160), (2050, 1040), (2049, 6176), (5, 30016)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["normal", "special"])
def test_rows(R, C, dtype, kind):
    say("int8 rows", R, C, dtype, kind)
    x = (special(R, C, R + C) if kind == "special" else normal((R, C), R + C)).to(dtype)
    x[x.isinf()] = 1.0  # (3e38 may become one in BF16)
    q, s = fq.quantize_int8(x.cuda())
    wq, ws = rule(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)


@pytest.mark.parametrize("R,C", [(1, 8), (16, 24), (17, 136), (127, 128), (129, 520), (2000, 264), (9000, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["normal", "special"])
def test_columns(R, C, dtype, kind):
    say("int8 columns", R, C, dtype, kind)
    x = (special(C, R, R + C).t() if kind == "special" and R > 3 else normal((R, C), R + C)).to(dtype).contiguous()
    x[x.isinf()] = 1.0
    qt, st = fq.quantize_int8_t(x.cuda())
    wq, ws = rule(x.t())
    assert torch.equal(st.cpu(), ws)
    assert torch.equal(qt.cpu()[:, :R], wq) and not qt.cpu()[:, R:].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_and_infinity_mark_their_row(dtype):
    say("int8 nan", dtype)
    x = normal((40, 64), 3, dtype)
    x[3, 40], x[7, 5], x[9, 63] = float("nan"), float("inf"), -float("inf")
    q, s = fq.quantize_int8(x.cuda())
    qt, st = fq.quantize_int8_t(x.cuda())
    assert s.isnan().nonzero().flatten().tolist() == [3, 7, 9]
    assert st.isnan().nonzero().flatten().tolist() == [5, 40, 63]
    w, sw = codes((24, 64), 4).cuda(), scales(24, 5).cuda()
    for rows in (slice(0, 8), slice(0, 40)):
        y = fq.linear_int8(x.cuda()[rows], w, sw)
        bad = y.isnan()
        assert bad.all(1).nonzero().flatten().tolist() == [r for r in (3, 7, 9) if r < rows.stop]
        assert bad.any(1).equal(bad.all(1))


def test_strides_and_guards():
    say("int8 strides")
    R, C = 70, 96
    big = normal((R, C + 40), 6, BF16).cuda()
    x = big[:, 8:C + 8]
    qg = torch.full((R + 2, C + 32), 9, dtype=torch.int8, device="cuda")
    sg = torch.full((R + 3,), 9.0, device="cuda")
    fq.fp8bq_quantize_int8(x, qg[:R, :C], sg[:R])
    tg = torch.full((C + 2, 112), 9, dtype=torch.int8, device="cuda")
    ug = torch.full((C + 3,), 9.0, device="cuda")
    ws = torch.empty(fq.fp8bq_quantize_int8_t_workspace_size(R, C), dtype=torch.uint8, device="cuda")
    fq.fp8bq_quantize_int8_t(x, tg[:C, :80], ug[:C], ws)
    wq, wsc = rule(x.cpu())
    tq, tsc = rule(x.cpu().t())
    assert torch.equal(qg[:R, :C].cpu(), wq) and torch.equal(sg[:R].cpu(), wsc)
    assert torch.equal(tg[:C, :R].cpu(), tq) and torch.equal(ug[:C].cpu(), tsc) and not tg[:C, R:80].any()
    for whole, part in ((qg, qg[:R, :C]), (tg, tg[:C, :80]), (sg, sg[:R]), (ug, ug[:C])):
        part.fill_(9)
        assert bool((whole == 9).all())


# one row to many, and on the tiles of 64, 128 and 256; contractions that end inside a stage and inside a step; N odd
SIZES = [(1, 1, 16), (1, 2048, 2048), (3, 77, 144), (9, 513, 1040), (16, 30000, 272), (16, 256, 8208), (17, 33, 16),
         (65, 130, 144), (300, 71, 2064), (777, 2560, 528), (1111, 1023, 4096), (4099, 4000, 400), (40, 64, 20000)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", [BF16, F32])
def test_gemm(M, N, K, out):
    say("int8 gemm", M, N, K, out)
    a, b, sa, sb = codes((M, K), M, -128), codes((N, K), N, -128), scales(M, 1), scales(N, 2)
    close(fq.gemm_int8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=out), exact(a, sa, b, sb))


@pytest.mark.parametrize("M,N,K", [(5, 96, 272), (300, 71, 2064), (64, 64, 20000)])
def test_gemm_added_to_the_output(M, N, K):
    say("int8 accumulate", M, N, K)
    a, b, sa, sb = codes((M, K), M), codes((N, K), N), scales(M, 1), scales(N, 2)
    c0 = normal((M, N), 3, std=10.0).cuda()
    got = fq.gemm_int8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out=c0.clone(), accumulate=True)
    add = exact(a, sa, b, sb)
    want = c0.double() + add
    torch.cuda.synchronize()
    assert bool(((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + 3.02 * 2.0 ** -24 * add.abs()).all())


def test_gemm_largest_sums():
    say("int8 largest sums")
    K = (1 << 17) - 16
    a, b = torch.full((20, K), -128, dtype=torch.int8), torch.full((36, K), -128, dtype=torch.int8)
    b[1] = 127
    one = torch.ones
    want = exact(a, one(20), b, one(36))
    assert float(want.max()) == 16384.0 * K
    close(fq.gemm_int8(a.cuda(), one(20).cuda(), b.cuda(), one(36).cuda(), out_dtype=F32), want)
    close(fq.gemm_int8(a[:3].cuda(), one(3).cuda(), b.cuda(), one(36).cuda(), out_dtype=F32), want[:3])


def test_gemm_strided_and_odd_outputs():
    say("int8 strided outputs")
    for M, N, K in ((7, 45, 80), (200, 333, 160), (600, 700, 128)):
        a, b, sa, sb = codes((M, K + 16), 1), codes((N + 4, K + 48), 2), scales(M, 3), scales(N, 4)
        want = exact(a[:, :K], sa, b[:N, 16:K + 16], sb)
        for out in (BF16, F32):
            for pad in (0, 1, 3, 8):
                guard = torch.full((M + 2, N + pad), 7.0, dtype=out, device="cuda")
                y = guard[:M, :N]
                fq.gemm_int8(a.cuda()[:, :K], sa.cuda(), b.cuda()[:N, 16:K + 16], sb.cuda(), out=y)
                close(y, want)
                y.fill_(7.0)
                assert bool((guard == 7.0).all()), (M, N, out, pad)


def test_empty_contraction_and_empty_sizes():
    say("int8 empty")
    z = torch.zeros
    a, b = z((5, 0), dtype=torch.int8, device="cuda"), z((9, 0), dtype=torch.int8, device="cuda")
    out = torch.full((5, 9), 3.0, device="cuda")
    fq.gemm_int8(a, z(5, device="cuda"), b, z(9, device="cuda"), out=out, accumulate=True)
    assert bool((out == 3.0).all())
    fq.gemm_int8(a, z(5, device="cuda"), b, z(9, device="cuda"), out=out)
    assert bool((out == 0.0).all())
    assert fq.linear_int8(z((0, 64), device="cuda"), z((9, 64), dtype=torch.int8, device="cuda"), z(9, device="cuda")).shape == (0, 9)
    q, s = fq.quantize_int8(z((0, 64), device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 13, 16, 17, 100, 1000])
@pytest.mark.parametrize("N,K", [(96, 64), (1000, 2048), (80, 14352), (40000, 144)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_is_quantizer_and_product(M, N, K, dtype):
    say("int8 linear", M, N, K, dtype)
    x = (normal((M, K), M + N) * torch.logspace(-3, 3, M).unsqueeze(1)).to(dtype).cuda()
    w, sw = codes((N, K), 1).cuda(), scales(N, 2).cuda()
    q, s = fq.quantize_int8(x)
    for out in (BF16, F32):
        assert torch.equal(fq.linear_int8(x, w, sw, out_dtype=out), fq.gemm_int8(q, s, w, sw, out_dtype=out))
    close(fq.linear_int8(x, w, sw, out_dtype=F32), exact(q, s, w, sw))


COUNTS = [[1], [0, 0, 3, 0], [5, 0, 1, 9], [1] * 16, [0] * 60 + [2, 0, 0, 7], [64, 1, 0, 130, 257], [700, 0, 3, 1500, 256, 128],
          [40] * 64]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}of{sum(c)}")
@pytest.mark.parametrize("N,K", [(40, 48), (130, 272), (513, 1024)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped(counts, N, K, dtype):
    say("int8 grouped", counts[:8], N, K, dtype)
    E, before, after = len(counts), 2, 3  # rows that belong to no expert
    n = torch.tensor([before] + counts)
    off = n.cumsum(0).cuda()
    T = int(off[-1]) + after
    x = (normal((T, K), T) * torch.logspace(-2, 2, T).unsqueeze(1)).to(dtype).cuda()
    w, sw = codes((E * N, K), 1), scales(E * N, 2)
    q, s = fq.quantize_int8(x)
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    o = off.tolist()
    for e in range(E):
        want[o[e]:o[e + 1]] = exact(q[o[e]:o[e + 1]], s[o[e]:o[e + 1]], w[e * N:(e + 1) * N], sw[e * N:(e + 1) * N])
    for out in (BF16, F32):
        y1 = torch.full((T, N), 5.0, dtype=out, device="cuda")
        y2 = y1.clone()
        fq.grouped_gemm_int8(q, s, off, w.cuda(), sw.cuda(), out=y1)
        fq.grouped_linear_int8(x, off, w.cuda(), sw.cuda(), out=y2)
        close(y1[before:T - after], want[before:T - after])
        assert torch.equal(y1, y2)
        assert bool((y1[:before] == 5.0).all()) and bool((y1[T - after:] == 5.0).all())


def test_grouped_offsets_out_of_range_stay_inside():
    say("int8 bad offsets")
    T, N, K, E = 50, 64, 64, 4
    x, w, sw = normal((T, K), 1).cuda(), codes((E * N, K), 2).cuda(), scales(E * N, 3).cuda()
    for off in ([0, -5, 1 << 40, 3, 70], [60, 50, 40, 30, 20], [-(1 << 62)] * 5):
        y = torch.full((T + 1, N), 5.0, device="cuda")
        fq.grouped_linear_int8(x, torch.tensor(off).cuda(), w, sw, out=y[:T])
        torch.cuda.synchronize()
        assert bool((y[T] == 5.0).all())


@pytest.mark.parametrize("M,N,K", [(1, 2048, 2048), (300, 512, 2064), (40, 64, 20000)])
def test_captured_and_replayed(M, N, K):
    say("int8 graph", M, N, K)
    x = normal((M, K), 1, BF16).cuda()
    w, sw = codes((N, K), 2).cuda(), scales(N, 3).cuda()
    fq.linear_int8(x, w, sw)
    fq.quantize_int8_t(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fq.linear_int8(x, w, sw)
        qt, st = fq.quantize_int8_t(x)
    for seed in range(3):
        x.copy_(normal((M, K), 10 + seed, BF16))
        graph.replay()
        got = [t.clone() for t in (y, qt, st)]
        torch.cuda.synchronize()
        for a, b in zip(got, (fq.linear_int8(x, w, sw), *fq.quantize_int8_t(x))):
            assert torch.equal(a, b)


def test_a_layer_step():
    """Forward and both gradients as a training loop chains them."""
    say("int8 step")
    M, N, K = 1001, 272, 400
    x, w, dy = normal((M, K), 1, BF16), normal((N, K), 2, BF16, 0.02), normal((M, N), 3, BF16, 1e-3)
    qw, sw = fq.quantize_int8(w.cuda())
    y = fq.linear_int8(x.cuda(), qw, sw)
    dx = fq.gemm_int8(*fq.quantize_int8(dy.cuda()), *fq.quantize_int8_t(w.cuda()))
    dw = fq.gemm_int8(*fq.quantize_int8_t(dy.cuda()), *fq.quantize_int8_t(x.cuda()))
    (qx, sx), (qd, sd), (rw, tw) = rule(x), rule(dy), rule(w)
    (wt, swt), (dt, sdt), (xt, sxt) = rule(w.t()), rule(dy.t()), rule(x.t())
    close(y, exact(qx, sx, rw, tw))
    close(dx, exact(qd, sd, wt, swt))
    close(dw, exact(dt, sdt, xt, sxt))
