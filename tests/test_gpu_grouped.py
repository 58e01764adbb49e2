"""Products grouped by expert and their token-axis quantizer against the float64 oracle, one expert at a
time: codes and scales bit for bit; products within 1e-4 ||a|| ||b|| of the float64 result (the FP32 rule of
parity.py: the MFMA's sum of a 128-long block and the fold's FP32 rounding), and a BF16 output within half a
unit in its last place more, 2^-8 |y| (that sum may lie on the other side of a tie: with one or two tokens in
the contraction ties are common).  Sizes: experts without tokens (first, middle, last, all), one token, counts around 128 and around a tile, one
expert with everything, more experts than a wave has lanes, token buffers larger than the tokens,
strided operands and FP32 accumulation."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import oracle
import synth
from parity import F32_ABS, f32_bits, say, to_np_f64

pytestmark = pytest.mark.gpu

CASES = {
    "ragged": ([3, 0, 128, 129, 1, 260, 0], 256, 384),
    "first_empty": ([0, 77], 128, 128),
    "one_token": ([0, 0, 1, 0], 384, 256),
    "one_expert": ([333], 256, 128),
    "all_on_one": ([0, 0, 700, 0], 128, 512),
    "tile_edges": ([256, 255, 257, 64, 63, 65, 128, 127], 128, 256),
    "many_experts": ([(7 * e) % 5 for e in range(130)], 128, 128),
    "most_experts": ([e % 2 for e in range(512)], 128, 128),
}
FMTS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")]
F = {"e4m3": (fq.E4M3, oracle.E4M3), "e5m2": (fq.E5M2, oracle.E5M2)}


def make(counts, N, K, seed, dtype=torch.bfloat16, before=0, after=0):
    E, n = len(counts), sum(counts)
    T = before + n + after
    x = synth.random_bf16((T, K), seed, 1.0, outliers=True).to(dtype)
    dy = synth.random_bf16((T, N), seed + 1, 1e-3).to(dtype)
    w = synth.random_bf16((E * N, K), seed + 2, 0.02)
    off = before + np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    return x, dy, w, off


def dev(t):
    return t.to("cuda") if isinstance(t, torch.Tensor) else torch.from_numpy(np.asarray(t)).to("cuda")


def dequant_cols(x, fmt):
    """float64 values of the 128x1 codes of x [n, C], the rows padded with zeros to whole blocks."""
    n, C = x.shape
    xp = np.zeros(((n + 127) // 128 * 128, C), np.float32)
    xp[:n] = x
    q, s = oracle.quant_act_128x1(xp, fmt)
    return q, s, oracle.dequant_act_128x1(q, s, fmt)


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantizer_codes_and_scales(name, dtype):
    counts, N, K = CASES[name]
    say("grouped quantizer", name, dtype)
    x, _, _, off = make(counts, N, K, 10, dtype)
    fr, fc = fq.E4M3, fq.E5M2
    q, s, qt, st = fq.quantize_act_grouped_dual(dev(x), dev(off), fr, fc)
    qt2, st2 = fq.quantize_act_grouped_128x1(dev(x), dev(off), fc)
    torch.cuda.synchronize()
    xn = x.float().numpy()
    oq, os_ = oracle.quant_act_1x128(xn, oracle.E4M3)
    assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(f32_bits(s.cpu().numpy().T), f32_bits(os_))
    qt, st, qt2, st2 = (t.cpu().numpy() for t in (qt, st, qt2, st2))
    p = 0
    for e, n in enumerate(counts):
        b = (n + 127) // 128
        ocq, ocs, _ = dequant_cols(xn[off[e]:off[e + 1]], oracle.E5M2)
        for got_q, got_s in ((qt, st), (qt2, st2)):
            assert np.array_equal(got_q[:, p:p + 128 * b].T, ocq.reshape(128 * b, K)), (name, e)
            assert np.array_equal(f32_bits(got_s[p // 128:p // 128 + b]), f32_bits(ocs.reshape(b, K))), (name, e)
        p += 128 * b
    assert p <= qt.shape[1]


def check(got, a, b, f32, what):
    """got [I, J] against a [I, L] . b [J, L]^T in float64."""
    y = a @ b.T
    lim = F32_ABS * np.outer(np.linalg.norm(a, axis=1), np.linalg.norm(b, axis=1))
    if not f32:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y)
    off = np.abs(got - y) - lim
    assert np.all(off <= 0), f"{what}: {int((off > 0).sum())} of {off.size} outside"


def products(name, fdy, fx, out_dtype, seed=20, before=0, after=0):
    """Runs fprop, dgrad and wgrad and checks every expert's rows."""
    counts, N, K = CASES[name]
    E = len(counts)
    x, dy, w, off = make(counts, N, K, seed, before=before, after=after)
    (gdy, ody), (gx, ox) = F[fdy], F[fx]
    offd = dev(off)
    qw, sw, qwt = fq.quantize_weight_dual(dev(w), fq.E4M3)
    qx, sx, qxt, sxt = fq.quantize_act_grouped_dual(dev(x), offd, gx, gx)
    qdy, sdy, qdyt, sdyt = fq.quantize_act_grouped_dual(dev(dy), offd, gdy, gdy)
    T = x.shape[0]
    y = torch.full((T, N), 7.0, dtype=out_dtype, device="cuda")
    dx = torch.full((T, K), 7.0, dtype=out_dtype, device="cuda")
    fq.grouped_gemm_fprop(qx, sx, offd, qw, sw, gx, fq.E4M3, out=y)
    fq.grouped_gemm_dgrad(qdy, sdy, offd, qwt, sw, gdy, fq.E4M3, out=dx)
    dw = fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offd, gdy, gx, out_dtype=out_dtype)
    torch.cuda.synchronize()
    f32 = out_dtype == torch.float32
    oqw, osw = oracle.quant_weight_128x128(w.float().numpy(), oracle.E4M3)
    wd = oracle.dequant_weight_128x128(oqw, osw, oracle.E4M3).reshape(E, N, K)
    y, dx, dw = to_np_f64(y), to_np_f64(dx), to_np_f64(dw).reshape(E, N, K)
    for e, n in enumerate(counts):
        if n == 0:
            assert not dw[e].any(), (name, e)
            continue
        rows = slice(off[e], off[e + 1])
        xn, dyn = x.float().numpy()[rows], dy.float().numpy()[rows]
        xd = oracle.dequant_act_1x128(*oracle.quant_act_1x128(xn, ox), ox)
        dyd = oracle.dequant_act_1x128(*oracle.quant_act_1x128(dyn, ody), ody)
        check(y[rows], xd, wd[e], f32, f"{name} fprop {e}")
        check(dx[rows], dyd, wd[e].T, f32, f"{name} dgrad {e}")
        xc, dyc = dequant_cols(xn, ox)[2], dequant_cols(dyn, ody)[2]
        check(dw[e], dyc.T, xc.T, f32, f"{name} wgrad {e}")
    outside = np.r_[0:off[0], off[-1]:T]
    assert np.all(y[outside] == 7.0) and np.all(dx[outside] == 7.0)


@pytest.mark.parametrize("name", sorted(CASES))
def test_products(name):
    say("grouped products", name)
    products(name, "e4m3", "e4m3", torch.bfloat16)


@pytest.mark.parametrize("fdy,fx", FMTS)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_formats_and_output_types(fdy, fx, out_dtype):
    say("grouped formats", fdy, fx, out_dtype)
    products("ragged", fdy, fx, out_dtype, seed=40)


def test_rows_outside_every_expert_are_left_alone():
    say("grouped outside rows")
    products("ragged", "e4m3", "e4m3", torch.bfloat16, seed=60, before=5, after=131)


@pytest.mark.parametrize("share,N,K", [(300, 2048, 1408), (40, 512, 256), (1200, 256, 2048)])
def test_larger_products_take_every_tile_shape(share, N, K):
    """Sizes at which the planner takes its larger tiles; compared on the device in float64."""
    say("grouped larger", share, N, K)
    counts = [share, 2 * share + 13, 0, share // 2]
    E = len(counts)
    x, dy, w, off = make(counts, N, K, 80)
    x, dy, w, offd = dev(x), dev(dy), dev(w), dev(off)
    qw, sw, qwt = fq.quantize_weight_dual(w, fq.E4M3)
    qx, sx, qxt, sxt = fq.quantize_act_grouped_dual(x, offd)
    qdy, sdy, qdyt, sdyt = fq.quantize_act_grouped_dual(dy, offd)
    y = fq.grouped_gemm_fprop(qx, sx, offd, qw, sw)
    dx = fq.grouped_gemm_dgrad(qdy, sdy, offd, qwt, sw)
    dw = fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offd)
    torch.cuda.synchronize()

    def dec(q):
        return q.view(torch.float8_e4m3fn).double()

    wd = dec(qw) * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    xd, dyd = (dec(q) * s.double().t().repeat_interleave(128, 1) for q, s in ((qx, sx), (qdy, sdy)))
    p = 0
    for e, n in enumerate(counts):
        b = (n + 127) // 128
        rows, pad, we = slice(off[e], off[e + 1]), slice(p, p + 128 * b), wd[e * N:(e + 1) * N]
        p += 128 * b
        xc, dyc = (dec(q[:, pad]) * s[pad.start // 128:pad.stop // 128].double().t().repeat_interleave(128, 1)
                   for q, s in ((qxt, sxt), (qdyt, sdyt)))
        for got, a, bt, what in ((y[rows], xd[rows], we, "fprop"), (dx[rows], dyd[rows], we.t(), "dgrad"),
                                 (dw[e * N:(e + 1) * N], dyc, xc, "wgrad")):
            check(to_np_f64(got), a.cpu().numpy(), bt.cpu().numpy(), False, f"{what} {e}")


def test_accumulation_into_main_grads():
    say("grouped accumulate")
    counts, N, K = CASES["ragged"]
    E = len(counts)
    x, dy, _, off = make(counts, N, K, 90)
    offd = dev(off)
    qxt, sxt = fq.quantize_act_grouped_128x1(dev(x), offd)
    qdyt, sdyt = fq.quantize_act_grouped_128x1(dev(dy), offd)
    one = fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offd, out_dtype=torch.float32)
    acc = torch.randn(E * N, K, device="cuda")
    start = acc.clone()
    fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offd, out=acc, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(acc, start + one)  # one FP32 addition per element


def test_strided_operands_and_outputs():
    say("grouped strided")
    counts, N, K = CASES["ragged"]
    x, dy, w, off = make(counts, N, K, 100)
    T, E = x.shape[0], len(counts)
    offd = dev(off)

    def wide(t, extra):
        big = torch.zeros(t.shape[0], t.shape[1] + extra, dtype=t.dtype, device="cuda")
        big[:, :t.shape[1]] = t
        return big[:, :t.shape[1]]

    xs = wide(dev(x), 64)
    q, s, qt, st = fq.quantize_act_grouped_dual(xs, offd)
    q0, s0, qt0, st0 = fq.quantize_act_grouped_dual(dev(x), offd)
    qw, sw = fq.quantize_weight_128x128(dev(w), fq.E4M3)
    y = torch.zeros(T, N + 16, dtype=torch.bfloat16, device="cuda")
    fq.grouped_gemm_fprop(wide(q, 32), wide(s, 4 + -T % 4), offd, wide(qw, 48), sw, out=y[:, :N])
    y0 = fq.grouped_gemm_fprop(q0, s0, offd, qw, sw)
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and torch.equal(s, s0)
    assert torch.equal(y[:, :N], y0) and not y[:, N:].any()


@pytest.mark.parametrize("offsets", [[0, 90, 30, 1000, 64], [-5, 10, 20, 30, 64], [0, 2 ** 40, -2 ** 50, 7, 64]])
def test_offsets_out_of_order_stay_inside_the_matrices(offsets):
    """Offsets that do not ascend or point past the tokens give unspecified values, inside the outputs only:
    guard rows and columns around every output keep theirs."""
    say("grouped bad offsets", offsets)
    E, T, N, K = 4, 64, 128, 128
    x, dy, w, _ = make([16] * 4, N, K, 110)
    offd = dev(np.asarray(offsets, np.int64))
    padded = fq.fp8bq_grouped_padded_rows(T, E)
    qw, sw, qwt = fq.quantize_weight_dual(dev(w), fq.E4M3)

    def guarded(r, c, dtype):
        big = torch.full((r + 4, c + 16), 7, dtype=dtype, device="cuda")
        return big, big[2:r + 2, :c] if dtype != torch.float32 else big[4:r + 4, :c]

    outs = [guarded(T, K, torch.uint8), guarded(K // 128, T, torch.float32), guarded(K, padded, torch.uint8),
            guarded(padded // 128, K, torch.float32), guarded(T, N, torch.bfloat16), guarded(E * N, K, torch.bfloat16)]
    (_, q), (_, s), (_, qt), (_, st), (_, y), (_, dw) = outs
    fq.fp8bq_quantize_act_grouped(dev(x), offd, fq.E4M3, q, s, fq.E4M3, qt, st)
    fq.fp8bq_grouped_gemm_fprop(q, s, fq.E4M3, offd, qw, sw, fq.E4M3, y)
    qdyt, sdyt = fq.quantize_act_grouped_128x1(dev(dy), offd)
    fq.fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fq.E4M3, qt, st, fq.E4M3, offd, dw)
    torch.cuda.synchronize()
    for big, inner in outs:
        held = torch.ones_like(big, dtype=torch.bool)
        r0 = (inner.data_ptr() - big.data_ptr()) // big.element_size() // big.stride(0)
        held[r0:r0 + inner.shape[0], :inner.shape[1]] = False
        assert torch.all(big[held] == 7)


def test_gradients_match_differences():
    """On values FP8 holds exactly (-1, 0, 1 and a 7 in every group: scale 1/64), y_e = x_e w_e^T is bilinear: the change
    of sum(y dy) when one entry of x or w moves by h is h times its gradient, exactly (integers below 2^24)."""
    say("grouped differences")
    counts, N, K = [40, 0, 130, 1], 128, 256
    E, T = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    rng = np.random.default_rng(3)

    def exact(r, c):
        v = rng.integers(-1, 2, (r, c)).astype(np.float32)
        for i in range(r):  # a 7 in every 128 of a row, and (first row of a block of tokens, below) of a column
            v[i, (5 * i) % 128::128] = 7.0
        return v

    x, dy, w = exact(T, K), exact(T, N), exact(E * N, K)
    for e, n in enumerate(counts):
        for b in range(0, n, 128):
            x[off[e] + b], dy[off[e] + b] = 7.0, 7.0
    offd = dev(off)

    def run(x_, w_):
        qw, sw, qwt = fq.quantize_weight_dual(dev(w_), fq.E4M3)
        qx, sx = fq.quantize_act_1x128(dev(x_), fq.E4M3)
        y = fq.grouped_gemm_fprop(qx, sx, offd, qw, sw, out_dtype=torch.float32)
        return float((y.double() * dev(dy).double()).sum()), sw, qwt

    base, sw, qwt = run(x, w)
    qdy, sdy, qdyt, sdyt = fq.quantize_act_grouped_dual(dev(dy), offd)
    qxt, sxt = fq.quantize_act_grouped_128x1(dev(x), offd)
    dx = fq.grouped_gemm_dgrad(qdy, sdy, offd, qwt, sw, out_dtype=torch.float32).cpu().numpy()
    dw = fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, offd, out_dtype=torch.float32).cpu().numpy()
    for e in range(E):
        rows, we = slice(off[e], off[e + 1]), w[e * N:(e + 1) * N]
        assert np.array_equal(dx[rows], dy[rows] @ we)
        assert np.array_equal(dw[e * N:(e + 1) * N], dy[rows].T @ x[rows])
    for i, j in ((3, 7), (100, 200), (169, 1)):
        x2 = x.copy()
        h = -1.0 if x2[i, j] > 0 else 1.0
        assert x2[i, j] != 7.0
        x2[i, j] += h
        assert run(x2, w)[0] - base == h * dx[i, j]
    for n, k in ((5, 9), (2 * N + 64, 130), (3 * N + 127, 255)):
        w2 = w.copy()
        h = -1.0 if w2[n, k] > 0 else 1.0
        assert w2[n, k] != 7.0
        w2[n, k] += h
        assert run(x, w2)[0] - base == h * dw[n, k]


def test_no_tokens():
    say("grouped no tokens")
    E, N, K = 3, 128, 256
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    u8, f32 = torch.uint8, torch.float32
    dw = torch.full((E * N, K), 5.0, dtype=torch.bfloat16, device="cuda")
    e = lambda *s, d: torch.empty(s, dtype=d, device="cuda")
    fq.fp8bq_grouped_gemm_wgrad(e(N, 0, d=u8), e(0, N, d=f32), fq.E4M3, e(K, 0, d=u8), e(0, K, d=f32), fq.E4M3, off, dw)
    y = fq.grouped_gemm_fprop(e(0, K, d=u8), e(K // 128, 0, d=f32), off, e(E * N, K, d=u8), e(E, K // 128, d=f32))
    torch.cuda.synchronize()
    assert not dw.any() and y.shape == (0, N)


def test_graph_replays_and_other_streams():
    """A captured step replays to the eager result with new tokens and new offsets in the same buffers."""
    say("grouped graph")
    counts, N, K = CASES["ragged"]
    x, _, w, off = make(counts, N, K, 120)
    xd, offd = dev(x), dev(off)
    qw, sw = fq.quantize_weight_128x128(dev(w), fq.E4M3)

    def step():
        q, s, qt, st = fq.quantize_act_grouped_dual(xd, offd)
        return fq.grouped_gemm_fprop(q, s, offd, qw, sw), fq.grouped_gemm_wgrad(qt, st, qt, st, offd)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dw = step()
    T = x.shape[0]
    for i, cuts in enumerate(([0, 1, 2, 3, 300, 400, 500], [100] * 7, [10, 20, 30, 200, 200, 201, 500])):
        xd.copy_(synth.random_bf16(tuple(x.shape), 130 + i))
        offd.copy_(torch.tensor([0] + cuts[1:] + [T], dtype=torch.int64))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ye, dwe = step()
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(dw, dwe)
