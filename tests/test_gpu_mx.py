"""MXFP4 quantizer and products against the float64 oracle (oracle/mx.py).

Codes and scales bit for bit.  Products within 1e-4 ||a|| ||b|| of the float64 result (the FP32 rule of
parity.py), and a BF16 output within half a unit in its last place more, 2^-8 |y|."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import synth
from oracle import mx
from parity import F32_ABS, say, to_np_f64

pytestmark = pytest.mark.gpu


def dev(t):
    return t.to("cuda") if isinstance(t, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(t)).to("cuda")


def special(R, C, seed):
    """Random values with zeros, subnormals, ties, huge values, exact powers of two and signed zeros."""
    x = synth.random_f32((R, C), seed, 1.0).numpy()
    rng = np.random.default_rng(seed)
    flat = x.reshape(-1)
    pick = rng.integers(0, flat.size, flat.size // 3)
    flat[pick] = rng.choice(np.array([0.0, -0.0, 1e-40, -3e-45, 0.25, 0.75, 2.5, -3.5, 5.0, 6.0, 7.0, 1e30, -2.0 ** 100,
                                      2.0 ** -126, 2.0 ** -125, 1.5 * 2.0 ** -127], np.float32), pick.size)
    if R > 3:
        x[1] = 0.0
        x[2] = np.float32(1e-41) * rng.integers(-9, 9, C)
        x[3] *= np.float32(2.0 ** -120)
    return x


SHAPES = [(1, 32), (1, 128), (5, 96), (32, 256), (33, 160), (127, 288), (128, 128), (129, 416), (300, 2080)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "special"])
def test_quantizer_codes_and_scales(R, C, dtype, kind):
    say("mx quantizer", R, C, dtype, kind)
    x = torch.from_numpy(special(R, C, R + C)) if kind == "special" else synth.random_f32((R, C), R + C, 1.0)
    x = x.to(dtype)
    xn = x.float().numpy()
    xd = dev(x)
    q, s, qt, st = fq.quantize_mxfp4_dual(xd)
    q1, s1 = fq.quantize_mxfp4(xd)
    qt1, st1 = fq.quantize_mxfp4_t(xd)
    torch.cuda.synchronize()
    code, scale = mx.quant_mx_rows(xn)
    tcode, tscale = mx.quant_mx_rows(xn.T)
    for a, b in ((q, s), (q1, s1)):
        assert np.array_equal(b.cpu().numpy(), mx.scale_words(scale))
        assert np.array_equal(a.cpu().numpy(), mx.pack(code))
    for a, b in ((qt, st), (qt1, st1)):
        assert np.array_equal(b.cpu().numpy(), mx.scale_words(tscale))
        assert np.array_equal(a.cpu().numpy(), mx.pack(tcode))


def test_columns_of_any_eighth_width():
    say("mx quantizer narrow columns")
    x = synth.random_bf16((77, 40), 3)
    qt, st = fq.quantize_mxfp4_t(dev(x))
    tcode, tscale = mx.quant_mx_rows(x.float().numpy().T)
    assert np.array_equal(qt.cpu().numpy(), mx.pack(tcode))
    assert np.array_equal(st.cpu().numpy(), mx.scale_words(tscale))


def test_nan_and_infinity_mark_their_block():
    say("mx quantizer nan")
    x = synth.random_f32((64, 128), 5, 1.0)
    x[3, 40], x[7, 5], x[9, 127] = float("nan"), float("inf"), -float("inf")
    for dt in (torch.float32, torch.bfloat16):
        q, s, qt, st = fq.quantize_mxfp4_dual(dev(x.to(dt)))
        _, scale = mx.quant_mx_rows(x.to(dt).float().numpy())
        _, tscale = mx.quant_mx_rows(x.to(dt).float().numpy().T)
        assert np.array_equal(s.cpu().numpy(), mx.scale_words(scale)) and int((scale == 255).sum()) == 3
        assert np.array_equal(st.cpu().numpy(), mx.scale_words(tscale))


def test_strided_input_and_guarded_outputs():
    say("mx quantizer strides")
    R, C = 70, 96
    big = synth.random_bf16((R, C + 40), 6)
    x = dev(big)[:, :C]
    outs = [torch.full((R + 2, C // 2 + 16), 9, dtype=torch.uint8, device="cuda"),
            torch.full((3, R + 3, 4), 9, dtype=torch.uint8, device="cuda"),
            torch.full((C + 2, 64), 9, dtype=torch.uint8, device="cuda"),
            torch.full((3, C + 5, 4), 9, dtype=torch.uint8, device="cuda")]
    q, s = outs[0][:R, :C // 2], outs[1][:1, :R]
    qt, st = outs[2][:C, :48], outs[3][:1, :C]
    fq.fp8bq_quantize_mxfp4(x, q, s, qt, st)
    code, scale = mx.quant_mx_rows(big[:, :C].float().numpy())
    tcode, tscale = mx.quant_mx_rows(big[:, :C].float().numpy().T)
    assert np.array_equal(q.cpu().numpy(), mx.pack(code)) and np.array_equal(s.cpu().numpy(), mx.scale_words(scale))
    assert np.array_equal(qt.cpu().numpy(), mx.pack(tcode)) and np.array_equal(st.cpu().numpy(), mx.scale_words(tscale))
    for o, i in zip(outs, (q, s, qt, st)):
        i.fill_(9)
        assert torch.all(o == 9)


# -- products ----------------------------------------------------------------------------------

def check(got, a, b, f32, what):
    """got [I, J] against a [I, L] . b [J, L]^T in float64."""
    y = a @ b.T
    lim = F32_ABS * np.outer(np.linalg.norm(a, axis=1), np.linalg.norm(b, axis=1))
    if not f32:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y)
    off = np.abs(to_np_f64(got) - y) - lim
    assert np.all(off <= 0), f"{what}: {int((off > 0).sum())} of {off.size} outside"


def operand(R, K, seed, std=1.0, outliers=False):
    """Codes and scales on the device, and their float64 values."""
    x = synth.random_bf16((R, K), seed, std, outliers=outliers).float().numpy()
    code, scale = mx.quant_mx_rows(x)
    return dev(mx.pack(code)), dev(mx.scale_words(scale)), mx.mx_values(code, scale)


SIZES = [(1, 1, 32), (1, 16, 128), (3, 40, 96), (16, 17, 256), (17, 100, 160), (33, 129, 544), (64, 64, 512),
         (65, 250, 288), (100, 264, 2048), (129, 513, 352), (200, 300, 1120), (257, 259, 608), (400, 1000, 1312)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32", "accumulate"])
def test_gemm(M, N, K, out):
    say("mx gemm", M, N, K, out)
    qa, sa, a = operand(M, K, M + K, outliers=True)
    qb, sb, b = operand(N, K, N + K + 1, 0.02)
    if out == "accumulate":
        c = torch.randn(M, N, device="cuda")
        start = c.clone()
        one = fq.gemm_mxfp4(qa, sa, qb, sb, out_dtype=torch.float32)
        fq.gemm_mxfp4(qa, sa, qb, sb, out=c, accumulate=True)
        assert torch.equal(c, start + one)
        return
    y = fq.gemm_mxfp4(qa, sa, qb, sb, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    check(y, a, b, out == "f32", (M, N, K))


@pytest.mark.parametrize("M,N,K", [(512, 2048, 2080), (2048, 1000, 4096), (3000, 2560, 1024)])
def test_larger_products(M, N, K):
    say("mx gemm larger", M, N, K)
    qa, sa, a = operand(M, K, 7)
    qb, sb, b = operand(N, K, 8, 0.02)
    check(fq.gemm_mxfp4(qa, sa, qb, sb), a, b, False, (M, N, K))


@pytest.mark.parametrize("M,N,K", [(800, 1024, 160), (3000, 2560, 1024), (4096, 4100, 288)])
def test_full_tiles_in_every_output_type(M, N, K):
    """Tiles of every size away from the edges, in outputs with guard columns."""
    say("mx gemm outputs", M, N, K)
    qa, sa, a = operand(M, K, 17)
    qb, sb, b = operand(N, K, 18, 0.02)
    wide = torch.full((M, N + 12), 7.0, device="cuda")
    one = fq.gemm_mxfp4(qa, sa, qb, sb, out=wide[:, :N])
    check(one, a, b, True, (M, N, K))
    half = torch.full((M, N + 12), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.gemm_mxfp4(qa, sa, qb, sb, out=half[:, :N])
    assert torch.equal(half[:, :N], one.to(torch.bfloat16))
    start = torch.randn(M, N, device="cuda")
    acc = torch.full((M, N + 12), 7.0, device="cuda")
    acc[:, :N] = start
    fq.gemm_mxfp4(qa, sa, qb, sb, out=acc[:, :N], accumulate=True)
    assert torch.equal(acc[:, :N], start + one)
    for v in (wide, half, acc):
        assert torch.all(v[:, N:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (4, 33, 96), (13, 200, 5632), (16, 64, 128), (40, 130, 608),
                                   (700, 264, 544)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_quantizes_its_input(M, N, K, dtype):
    say("mx linear", M, N, K, dtype)
    x = synth.random_bf16((M, K), 11, 1.0, outliers=True).to(dtype)
    if dtype == torch.float32:
        x = x + torch.from_numpy(special(M, K, 12)).clamp(-1, 1) * 1e-3
    qw, sw, w = operand(N, K, 13, 0.02)
    xd = dev(x)
    y = fq.linear_mxfp4(xd, qw, sw, out_dtype=torch.float32)
    check(y, mx.mx_values(*mx.quant_mx_rows(x.numpy() if dtype == torch.float32 else x.float().numpy())), w, True,
          (M, N, K))
    q, s = fq.quantize_mxfp4(xd)
    two = fq.gemm_mxfp4(q, s, qw, sw, out_dtype=torch.float32)
    scale = float(two.abs().max())
    assert float((two - y).abs().max()) <= 1e-4 * scale


@pytest.mark.parametrize("M", [3, 90])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_takes_strided_rows(M, dtype):
    say("mx linear strided", M, dtype)
    N, K = 72, 256
    big = dev(synth.random_bf16((2 * M, K + 64), 15).to(dtype))
    qw, sw, _ = operand(2 * N, K, 16, 0.02)
    off = dev(np.array([0, M // 2, M], np.int64))
    for x in (big[:M, :K], big[::2, 32:K + 32]):
        want = fq.linear_mxfp4(x.contiguous(), qw, sw)
        assert torch.equal(fq.linear_mxfp4(x, qw, sw), want)
        assert torch.equal(fq.grouped_linear_mxfp4(x, off, qw, sw),
                           fq.grouped_linear_mxfp4(x.contiguous(), off, qw, sw))


def test_two_streams_do_not_share_state():
    """The same calls on two streams at once, each on its own tensors, give what they give one after the other."""
    say("mx two streams")
    N, K = 264, 544
    qw, sw, _ = operand(4 * N, K, 17, 0.02)
    xs = [dev(synth.random_bf16((200, K), 18 + i)) for i in range(2)]
    offs = [dev(np.array(o, np.int64)) for o in ([0, 3, 3, 100, 200], [0, 150, 151, 199, 200])]

    def step(i):
        q, s, qt, st = fq.quantize_mxfp4_dual(xs[i])
        return (fq.linear_mxfp4(xs[i], qw, sw), fq.gemm_mxfp4(qt, st, qt, st, out_dtype=torch.float32),
                fq.grouped_linear_mxfp4(xs[i], offs[i], qw, sw))

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_scales_over_the_whole_range():
    """Blocks from 2^-127 up: the scales multiply exactly."""
    say("mx scales")
    M, N, K = 20, 24, 256
    rng = np.random.default_rng(3)
    ca, cb = (rng.integers(0, 16, (r, K)).astype(np.uint8) for r in (M, N))
    ea = rng.integers(0, 120, (M, K // 32)).astype(np.uint8)
    eb = np.full((N, K // 32), 180, np.uint8)
    y = fq.gemm_mxfp4(dev(mx.pack(ca)), dev(mx.scale_words(ea)), dev(mx.pack(cb)), dev(mx.scale_words(eb)),
                      out_dtype=torch.float32)
    check(y, mx.mx_values(ca, ea), mx.mx_values(cb, eb), True, "scales")


@pytest.mark.parametrize("M", [5, 300])
def test_bytes_past_the_last_block_are_ignored_and_nan_blocks_reach_their_rows_only(M):
    say("mx nan", M)
    N, K = 70, 160
    qa, sa, a = operand(M, K, 21)
    qb, sb, b = operand(N, K, 22)
    want = fq.gemm_mxfp4(qa, sa, qb, sb, out_dtype=torch.float32)
    sa2, sb2 = sa.clone(), sb.clone()
    sa2[1, :, 1:], sb2[1, :, 1:] = 255, 255
    assert torch.equal(fq.gemm_mxfp4(qa, sa2, qb, sb2, out_dtype=torch.float32), want)
    sa2[0, 3, 2], sb2[1, 9, 0] = 255, 255
    y = fq.gemm_mxfp4(qa, sa2, qb, sb2, out_dtype=torch.float32)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[3], nan[:, 9] = True, True
    assert torch.equal(torch.isnan(y), nan) and torch.equal(y[~nan], want[~nan])
    x = synth.random_bf16((M, K), 23)
    x[2, 33] = float("inf")
    y = fq.linear_mxfp4(dev(x), qb, sb)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[2] = True
    assert torch.equal(torch.isnan(y), nan)


def test_strided_operands_and_outputs_stay_inside():
    say("mx strides")
    for M, N, K in ((9, 37, 96), (150, 203, 320)):
        qa, sa, a = operand(M, K, 31)
        qb, sb, b = operand(N, K, 32)

        def wide(t, extra):
            big = torch.full((t.shape[0], t.shape[1] + extra), 0xEE, dtype=torch.uint8, device="cuda")
            big[:, :t.shape[1]] = t
            return big[:, :t.shape[1]]

        def words(s, extra):
            big = torch.full((s.shape[0], s.shape[1] + extra, 4), 0xFF, dtype=torch.uint8, device="cuda")
            big[:, :s.shape[1]] = s
            return big[:, :s.shape[1]]

        for dt, pad in ((torch.bfloat16, 3), (torch.float32, 5), (torch.bfloat16, 8)):
            big = torch.full((M + 2, N + pad), 7.0, dtype=dt, device="cuda")
            fq.gemm_mxfp4(wide(qa, 16), words(sa, 3), wide(qb, 48), words(sb, 1), out=big[:M, :N])
            want = fq.gemm_mxfp4(qa, sa, qb, sb, out_dtype=dt)
            assert torch.equal(big[:M, :N], want)
            big[:M, :N] = 7.0
            assert torch.all(big == 7.0)


def test_empty_contraction_and_sizes():
    say("mx empty")
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    y = torch.full((5, 7), 3.0, device="cuda")
    fq.gemm_mxfp4(e(5, 0), e(0, 5, 4), e(7, 0), e(0, 7, 4), out=y, accumulate=True)
    assert torch.all(y == 3.0)
    fq.gemm_mxfp4(e(5, 0), e(0, 5, 4), e(7, 0), e(0, 7, 4), out=y)
    assert not y.any()
    assert fq.gemm_mxfp4(e(0, 32), e(1, 0, 4), e(7, 32), e(1, 7, 4)).shape == (0, 7)
    q, s, qt, st = fq.quantize_mxfp4_dual(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 32) and qt.shape == (64, 0)


GROUPS = {
    "decode": ([1, 0, 0, 1, 0, 1, 1, 0], 200, 2048),
    "ragged": ([3, 0, 40, 17, 1, 60, 0], 130, 544),
    "one_token": ([0, 0, 1], 33, 96),
    "many": ([(5 * e) % 7 for e in range(200)], 24, 160),
    "large": ([300, 0, 513, 128, 5], 520, 608),
    "most_experts": ([e % 3 for e in range(512)], 8, 64),
}


@pytest.mark.parametrize("name", sorted(GROUPS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped(name, dtype):
    counts, N, K = GROUPS[name]
    say("mx grouped", name, dtype)
    E, before, after = len(counts), 2, 3
    off = before + np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    T = int(off[-1]) + after
    x = synth.random_bf16((T, K), 41, 1.0, outliers=True).to(dtype)
    qw, sw, w = operand(E * N, K, 42, 0.02)
    xd, offd = dev(x), dev(off)
    y = torch.full((T, N), 7.0, device="cuda")
    fq.grouped_linear_mxfp4(xd, offd, qw, sw, out=y)
    q, s = fq.quantize_mxfp4(xd)
    y2 = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.grouped_gemm_mxfp4(q, s, offd, qw, sw, out=y2)
    torch.cuda.synchronize()
    v = mx.mx_values(*mx.quant_mx_rows(x.float().numpy()))
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        if rows.start < rows.stop:
            check(y[rows], v[rows], w[e * N:(e + 1) * N], True, (name, e))
            check(y2[rows], v[rows], w[e * N:(e + 1) * N], False, (name, e))
    outside = np.r_[0:before, T - after:T]
    assert torch.all(y[outside] == 7.0) and torch.all(y2[outside] == 7.0)


def test_gradients_match_differences():
    """On values the format holds exactly, y = x w^T is bilinear: the change of sum(y dy) when one entry of x or w
    moves by h is h times the gradient, exactly."""
    say("mx differences")
    M, N, K = 40, 72, 64
    rng = np.random.default_rng(5)

    def exact(r, c):  # multiples of 1/2 up to 2 with a 6 in every block of 32 either way: scale 1
        v = rng.integers(-4, 5, (r, c)).astype(np.float32) / 2
        for i in range(r):
            v[i, i % 32::32] = 6.0
        return v

    x, w, dy = exact(M, K), exact(N, K), exact(M, N)

    def loss(x_, w_):
        qw, sw = fq.quantize_mxfp4(dev(w_))
        y = fq.linear_mxfp4(dev(x_), qw, sw, out_dtype=torch.float32)
        return float((y.double() * dev(dy).double()).sum())

    pad = np.zeros((M, 96), np.float32)  # dgrad contracts over N: blocks of 32
    pad[:, :N] = dy
    wpad = np.zeros((96, K), np.float32)
    wpad[:N] = w
    qdy, sdy = fq.quantize_mxfp4(dev(pad))
    qwt, swt = fq.quantize_mxfp4_t(dev(wpad))
    dx = fq.gemm_mxfp4(qdy, sdy, qwt, swt, out_dtype=torch.float32).cpu().numpy()
    qdyt, sdyt = fq.quantize_mxfp4_t(dev(dy))
    qxt, sxt = fq.quantize_mxfp4_t(dev(x))
    dw = fq.gemm_mxfp4(qdyt, sdyt, qxt, sxt, out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x)  # sums of quarters below 2^22: exact
    base = loss(x, w)
    for i, j in ((0, 5), (17, 40), (39, 63)):
        h = 0.5 if x[i, j] < 1 else -0.5
        x2 = x.copy()
        x2[i, j] += h
        if x[i, j] != 6.0:
            assert loss(x2, w) - base == h * dx[i, j]
        h = 0.5 if w[i, j] < 1 else -0.5
        w2 = w.copy()
        w2[i, j] += h
        if w[i, j] != 6.0:
            assert loss(x, w2) - base == h * dw[i, j]


def test_graph_replays_and_other_streams():
    say("mx graph")
    M, N, K = 48, 136, 256
    qw, sw, _ = operand(N, K, 51)
    x = dev(synth.random_bf16((M, K), 52))
    off = dev(np.array([0, 10, 10, 48], np.int64))
    qe, se, _ = operand(3 * 40, K, 53)

    def step():
        q, s, qt, st = fq.quantize_mxfp4_dual(x)
        return (fq.linear_mxfp4(x[:5], qw, sw), fq.gemm_mxfp4(q, s, qw, sw), fq.gemm_mxfp4(qt, st, qt, st),
                fq.grouped_linear_mxfp4(x, off, qe, se))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(synth.random_bf16((M, K), 60 + i))
        off[1:3] = 5 + 13 * i
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
