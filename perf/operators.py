"""Measured cases of the microscaled 4-bit linear layer and of the expert-grouped FP8 linear layer.

Five operators, on the sizes of a 2B-class decoder (hidden 2048, QKV 2560, SwiGLU 2 x 5632) and of
experts cut from its feed-forward layer (1408 = 5632 / 4 wide):

  mx_forward      y = Q(x) . Wq^T, weights kept in 4 bits, x quantized in the call
  mx_backward     dx = Q(dy) . Q(W^T)^T and dw = Q(dy^T) . Q(x^T)^T, all operands in 4 bits
  expert_forward  y_e = Q(x_e) . Wq_e^T for the tokens of each expert (FP8, ragged groups)
  expert_backward dx_e = Q(dy_e) . Wq_e and dw_e = Q(dy_e^T) . Q(x_e^T)^T (FP8, ragged groups)
  expert_mx       y_e = Q(x_e) . Wq_e^T with the experts kept in 4 bits (serving)

4-bit operands: values of E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives, two per byte, the even
element in the low half) in blocks of 32 along the contraction, each block with a power-of-two scale
2^(b - 127): b - 127 = floor(log2(amax)) - 2, at least -127; elements round to the nearest, ties to
even, and saturate at 6.  FP8 operands: groups of 128 (blocks of 128 x 128 for weights) with scale
max(fp32(amax / fmt_max), 1e-12), codes of fp32(x / scale) rounded to the nearest, ties to even.

Tokens are sorted by expert; `offsets` (E + 1 int64 on the device) holds where each expert's begin.
The experts' weights are stacked, [E N, K].
"""

import torch

own = False

BF16 = torch.bfloat16
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one token through gate+up: the decode step of one sequence
        dict(name="mx_forward_1", op="mx_forward", M=1, N=11264, K=2048, x="bf16"),
        # a small odd batch of decoding sequences through the down projection
        dict(name="mx_forward_13", op="mx_forward", M=13, N=2048, K=5632, x="bf16"),
        # a short prompt (odd length, FP32 activations) through QKV
        dict(name="mx_forward_777", op="mx_forward", M=777, N=2560, K=2048, x="f32"),
        # a training micro-batch through gate+up: the largest product
        dict(name="mx_forward_16384", op="mx_forward", M=16384, N=11264, K=2048, x="bf16"),
        # backward of a small micro-batch; the tokens and the width end inside a block and a tile
        dict(name="mx_backward_1001", op="mx_backward", M=1001, N=2048, K=2080, x="bf16"),
        # backward of the down projection at a full micro-batch
        dict(name="mx_backward_16384", op="mx_backward", M=16384, N=2048, K=5632, x="bf16"),
        # few tokens on 8 experts, three of them idle: latency
        dict(name="expert_forward_77", op="expert_forward", E=8, T=77, N=2816, K=2048, skew=3.0),
        # a training micro-batch, two experts a token, on 64 uneven experts
        dict(name="expert_forward_32768", op="expert_forward", E=64, T=32768, N=2816, K=2048, skew=0.4),
        # backward of a small ragged batch
        dict(name="expert_backward_1001", op="expert_backward", E=8, T=1001, N=2048, K=1408, skew=1.0, dy_fmt="e4m3"),
        # backward of a training micro-batch with E5M2 gradients
        dict(name="expert_backward_32768", op="expert_backward", E=32, T=32768, N=2048, K=1408, skew=0.4, dy_fmt="e5m2"),
        # one token, six experts of 64: the decode step
        dict(name="expert_mx_6", op="expert_mx", E=64, T=6, N=2816, K=2048, skew=0.0),
        # 128 decoding sequences, six experts each
        dict(name="expert_mx_768", op="expert_mx", E=64, T=768, N=2816, K=2048, skew=0.4),
    ]


MOST_FLOPS = 2.0 * 16384 * 11264 * 2048


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("mx_forward", "mx_backward", "expert_forward", "expert_backward", "expert_mx"))
    while True:
        if op == "mx_forward":
            c = dict(op=op, M=_log(rng, 1, 16384), N=8 * _log(rng, 32, 1408), K=32 * _log(rng, 8, 352),
                     x=rng.choice(("bf16", "bf16", "f32")))
        elif op == "mx_backward":
            c = dict(op=op, M=_log(rng, 64, 16384), N=32 * _log(rng, 8, 176), K=32 * _log(rng, 8, 176), x="bf16")
        elif op == "expert_forward":
            c = dict(op=op, E=_log(rng, 1, 64), T=_log(rng, 1, 32768), N=128 * _log(rng, 2, 44), K=128 * _log(rng, 2, 22),
                     skew=rng.choice((0.0, 0.4, 1.0, 2.0)))
        elif op == "expert_backward":
            c = dict(op=op, E=_log(rng, 1, 32), T=_log(rng, 64, 32768), N=128 * _log(rng, 2, 22),
                     K=128 * _log(rng, 2, 22), skew=rng.choice((0.0, 0.4, 1.0, 2.0)), dy_fmt=rng.choice(("e4m3", "e5m2")))
        else:
            c = dict(op=op, E=_log(rng, 4, 64), T=_log(rng, 1, 4096), N=8 * _log(rng, 32, 352), K=32 * _log(rng, 8, 88),
                     skew=rng.choice((0.0, 0.4, 1.0)))
        # the products, and the padded token arrays that a plain form builds, stay under the largest listed case
        most = c["E"] * max(_counts(c)) if "E" in c else 0
        if work(c)["flops"] <= MOST_FLOPS / 2 and most * max(c["N"], c["K"]) <= 64 * 2048 * 2816:
            return c


def _counts(case):
    """Tokens per expert, most first: shares proportional to rank^-skew, largest remainders rounded up."""
    E, T = case["E"], case["T"]
    share = [(e + 1.0) ** -case["skew"] for e in range(E)]
    total = sum(share)
    exact_ = [T * s / total for s in share]
    n = [int(v) for v in exact_]
    left = sorted(range(E), key=lambda e: (n[e] - exact_[e], e))[:T - sum(n)]
    return [n[e] + (e in left) for e in range(E)]


def work(case):
    op = case["op"]
    N, K = case["N"], case["K"]
    if op == "mx_forward":
        M, xb = case["M"], 2 if case["x"] == "bf16" else 4
        return dict(bytes=M * K * xb + N * K * (0.5 + 1 / 32) + 2 * M * N, flops=2.0 * M * N * K)
    if op == "mx_backward":  # dy, x and W^T in; dx and dw out
        M = case["M"]
        return dict(bytes=2 * M * N + 2 * M * K + N * K * (0.5 + 1 / 32) + 2 * M * K + 2 * N * K, flops=4.0 * M * N * K)
    T, E = case["T"], case["E"]
    used = sum(n > 0 for n in _counts(case))
    if op == "expert_backward":
        return dict(bytes=2 * T * N + 2 * T * K + used * N * K + 2 * T * K + 2 * E * N * K, flops=4.0 * T * N * K)
    wb = 1.0 if op == "expert_forward" else 0.5 + 1 / 32
    return dict(bytes=2 * T * K + used * N * K * wb + 2 * T * N, flops=2.0 * T * N * K)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _normal(g, shape, std, outliers=False):
    t = torch.randn(shape, generator=g, device="cuda") * std
    if outliers:  # a hundredth of the channels fifty times larger
        t[:, torch.randperm(shape[1], generator=g, device="cuda")[:shape[1] // 100]] *= 50.0
    return t


def _pad_last(t, to):
    return t if t.shape[-1] == to else torch.cat([t, t.new_zeros(t.shape[:-1] + (to - t.shape[-1],))], -1)


def _on(t, v):
    """v as a tensor on t's device: a division by a Python number is a product with its rounded reciprocal there."""
    return torch.full((), v, dtype=torch.float32, device=t.device)


def _round_up(n, m):
    return -(-n // m) * m


def _to_fp4(w):
    """Packed codes [R, C/2] and scales [ceil(C/128), R, 4] of w [R, C], C a multiple of 32."""
    R, C = w.shape
    b = w.float().view(R, C // 32, 32)
    e = (torch.frexp(b.abs().amax(-1))[1] - 3).clamp(min=-127)
    y = torch.ldexp(b, -e.unsqueeze(-1)).view(R, C)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    a = y.abs().contiguous()
    # a tie goes to the even code: up from 0.75, 1.75 and 3.5, down from the others
    up, down = torch.bucketize(a, mids, right=True), torch.bucketize(a, mids)
    code = torch.where(up % 2 == 0, up, down).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    s = _pad_last((e + 127).to(torch.uint8), _round_up(C // 32, 4))
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(R, -1, 4).permute(1, 0, 2).contiguous()


def _to_fp8_blocks(w):
    """E4M3 codes [N, K] (uint8) and scales [N/128, K/128] of w, one scale for each 128 x 128 block."""
    N, K = w.shape
    b = w.float().view(N // 128, 128, K // 128, 128)
    s = (b.abs().amax((1, 3)) / _on(w, E4M3_MAX)).clamp(min=1e-12)
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(N, K).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, N, K = case["op"], case["N"], case["K"]
    s = dict(case)
    if op == "mx_forward":
        s["x"] = _normal(g, (case["M"], K), 1.0, True).to(BF16 if case["x"] == "bf16" else torch.float32)
        s["qw"], s["sw"] = _to_fp4(_normal(g, (N, K), 0.02).to(BF16))
    elif op == "mx_backward":
        s["x"] = _normal(g, (case["M"], K), 1.0, True).to(BF16)
        s["dy"] = _normal(g, (case["M"], N), 1e-3).to(BF16)
        s["qwt"], s["swt"] = _to_fp4(_normal(g, (K, N), 0.02).to(BF16))
    else:
        E, T = case["E"], case["T"]
        n = torch.tensor(_counts(case), device="cuda")[torch.randperm(E, generator=g, device="cuda")]
        s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)])
        s["x"] = _normal(g, (T, K), 1.0, True).to(BF16)
        w = _normal(g, (E * N, K), 0.02).to(BF16)
        if op == "expert_mx":
            s["qw"], s["sw"] = _to_fp4(w)
        else:
            s["qw"], s["sw"] = _to_fp8_blocks(w)
        if op == "expert_backward":
            s["dy"] = _normal(g, (T, N), 1e-3).to(BF16)
            s["qwt"] = s.pop("qw").t().contiguous()
    return s


# ---------------------------------------------------------------------------------------------
# the plain form: elementary operations in 32 bits
# ---------------------------------------------------------------------------------------------

def _fp4_rounded(x):
    """What the 4-bit codes of x stand for, blocks of 32 along the last axis (padded with zeros)."""
    C = x.shape[-1]
    b = _pad_last(x.float(), _round_up(C, 32)).unflatten(-1, (-1, 32))
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3).clamp(min=-127)
    y = torch.ldexp(b, -e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), y)
    return torch.ldexp(r, e).flatten(-2)[..., :C]


def _fp4_decoded(q, s):
    """Values [..., C] of packed codes [..., C/2] whose scales are [..., C/32] bytes."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 32))
    return torch.ldexp(v, s.int().unsqueeze(-1) - 127).flatten(-2)


def _fp8_rounded(x, fmt="e4m3"):
    """What the FP8 codes of x stand for, groups of 128 along the last axis."""
    top, kind = (E4M3_MAX, torch.float8_e4m3fn) if fmt == "e4m3" else (E5M2_MAX, torch.float8_e5m2)
    b = x.float().unflatten(-1, (-1, 128))
    s = (b.abs().amax(-1, keepdim=True) / _on(b, top)).clamp(min=1e-12)
    return ((b / s).clamp(-top, top).to(kind).float() * s).flatten(-2)


def _plain(s):
    op, N, K = s["op"], s["N"], s["K"]
    if op == "mx_forward":
        w = _fp4_decoded(s["qw"], s["sw"].permute(1, 0, 2).reshape(N, -1)[:, :K // 32])
        return (_fp4_rounded(s["x"]) @ w.t()).to(BF16)
    if op == "mx_backward":
        wt = _fp4_decoded(s["qwt"], s["swt"].permute(1, 0, 2).reshape(K, -1)[:, :N // 32])
        dx = _fp4_rounded(s["dy"]) @ wt.t()
        dw = _fp4_rounded(s["dy"].t()) @ _fp4_rounded(s["x"].t()).t()
        return dx.to(BF16), dw.to(BF16)

    # tokens laid out as [experts in use, most tokens of one, width], zeros where an expert has fewer
    E, off = s["E"], s["offsets"]
    n = off[1:] - off[:-1]
    used = n.nonzero().squeeze(1)
    cap = int(n.max())
    cap = _round_up(cap, 128) if op == "expert_backward" else cap
    place = torch.arange(cap, device=off.device)
    rows = off[used].unsqueeze(1) + place
    held = place < n[used].unsqueeze(1)
    rows = torch.where(held, rows, 0)

    def spread(t):
        return torch.where(held.unsqueeze(-1), t[rows], 0)

    if op == "expert_backward":
        w = s["qwt"].view(K, E, N).permute(1, 2, 0)[used].view(torch.float8_e4m3fn).float()
    elif op == "expert_forward":
        w = s["qw"].view(E, N, K)[used].view(torch.float8_e4m3fn).float()
    if op == "expert_mx":
        sw = s["sw"].permute(1, 0, 2).reshape(E, N, -1)[used, :, :K // 32]
        w = _fp4_decoded(s["qw"].view(E, N, K // 2)[used], sw)
        return torch.bmm(_fp4_rounded(spread(s["x"])), w.transpose(1, 2))[held].to(BF16)
    sw = s["sw"].view(E, N // 128, 1, K // 128, 1)[used]
    w = (w.unflatten(1, (-1, 128)).unflatten(3, (-1, 128)) * sw).flatten(3).flatten(1, 2)
    if op == "expert_forward":
        return torch.bmm(_fp8_rounded(spread(s["x"])), w.transpose(1, 2))[held].to(BF16)
    x, dy = spread(s["x"]), spread(s["dy"])
    dx = torch.bmm(_fp8_rounded(dy, s["dy_fmt"]), w)[held]
    dw = torch.zeros(E, N, K, device=off.device)
    dw[used] = torch.bmm(_fp8_rounded(dy.transpose(1, 2).contiguous(), s["dy_fmt"]),
                         _fp8_rounded(x.transpose(1, 2).contiguous()).transpose(1, 2).contiguous())
    return dx.to(BF16), dw.view(E * N, K).to(BF16)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_blockwise_quantized_amd as fq
    op = s["op"]
    if op == "mx_forward":
        return fq.linear_mxfp4(s["x"], s["qw"], s["sw"])
    if op == "mx_backward":
        qdy, sdy, qdyt, sdyt = fq.quantize_mxfp4_dual(s["dy"])
        qxt, sxt = fq.quantize_mxfp4_t(s["x"])
        return fq.gemm_mxfp4(qdy, sdy, s["qwt"], s["swt"]), fq.gemm_mxfp4(qdyt, sdyt, qxt, sxt)
    if op == "expert_mx":
        return fq.grouped_linear_mxfp4(s["x"], s["offsets"], s["qw"], s["sw"])
    if op == "expert_forward":
        q, sc = fq.quantize_act_1x128(s["x"])
        return fq.grouped_gemm_fprop(q, sc, s["offsets"], s["qw"], s["sw"])
    f = fq.E4M3 if s["dy_fmt"] == "e4m3" else fq.E5M2
    qdy, sdy, qdyt, sdyt = fq.quantize_act_grouped_dual(s["dy"], s["offsets"], f, f)
    qxt, sxt = fq.quantize_act_grouped_128x1(s["x"], s["offsets"])
    return (fq.grouped_gemm_dgrad(qdy, sdy, s["offsets"], s["qwt"], s["sw"], fdy=f),
            fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, s["offsets"], fdy=f))


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_fp4(x):
    """Nearest of the sixteen values times the block's scale, by comparing distances; x [R, C]."""
    R, C = x.shape
    v = torch.zeros(R, _round_up(C, 32), dtype=torch.float64, device=x.device)
    v[:, :C] = x.double()
    v = v.view(-1, 32)
    top = v.abs().max(1, keepdim=True).values
    scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -200))) - 2).clamp(min=2.0 ** -127)
    a = v.abs() / scale
    best = torch.zeros_like(a)
    for i, level in enumerate(E2M1[1:], 1):  # a nearer level wins; at equal distance an even code does
        far, near = (a - best).abs(), (a - level).abs()
        best = torch.where((near < far) | ((near == far) & (i % 2 == 0)), torch.full_like(a, level), best)
    return (torch.where(v < 0, -best, best) * scale).view(R, -1)[:, :C]


def _exact_fp4_codes(q, s):
    R = q.shape[0]
    m, d = (q & 7).long(), (q >> 4 & 7).long()
    lut = torch.tensor(E2M1, dtype=torch.float64, device=q.device)
    lo = lut[m] * torch.where(q & 8 > 0, -1.0, 1.0).double()
    hi = lut[d] * torch.where(q & 128 > 0, -1.0, 1.0).double()
    v = torch.empty(R, 2 * q.shape[1], dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = lo, hi
    scale = torch.exp2(s.transpose(0, 1).reshape(R, -1).double() - 127)[:, :v.shape[1] // 32]
    return v * scale.repeat_interleave(32, 1)


def _exact_fp8(x, fmt="e4m3"):
    """x [R, C], groups of 128 along C (the last may be shorter); the scale and the quotient are 32-bit values."""
    R, C = x.shape
    v = torch.zeros(R, _round_up(C, 128), dtype=torch.float64, device=x.device)
    v[:, :C] = x.double()
    v = v.view(-1, 128)
    top, bits, low = (448.0, 3, -6) if fmt == "e4m3" else (57344.0, 2, -14)
    scale = torch.maximum((v.abs().max(1, keepdim=True).values / _on(v, top).double()).float(), torch.tensor(1e-12, device=x.device)).double()
    y = (v / scale).float().double().clamp(-top, top)
    exp = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** (low - 1)))).clamp(min=low)
    ulp = torch.exp2(exp - bits)
    return ((torch.round(y / ulp) * ulp).clamp(-top, top) * scale).view(R, -1)[:, :C]


def _exact_blocks(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, N, K = s["op"], s["N"], s["K"]
    if op == "mx_forward":
        return _exact_fp4(s["x"]) @ _exact_fp4_codes(s["qw"], s["sw"]).t()
    if op == "mx_backward":
        dx = _exact_fp4(s["dy"]) @ _exact_fp4_codes(s["qwt"], s["swt"]).t()
        return dx, _exact_fp4(s["dy"].t()) @ _exact_fp4(s["x"].t()).t()
    off = s["offsets"].tolist()
    E, T = s["E"], s["T"]
    y = torch.zeros(T, K if op == "expert_backward" else N, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda") if op == "expert_backward" else None
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = s["x"][a:b]
        if op == "expert_mx":
            y[a:b] = _exact_fp4(x) @ _exact_fp4_codes(s["qw"][e * N:(e + 1) * N], s["sw"][:, e * N:(e + 1) * N]).t()
            continue
        sw = s["sw"][e * (N // 128):(e + 1) * (N // 128)]
        if op == "expert_forward":
            y[a:b] = _exact_fp8(x) @ _exact_blocks(s["qw"][e * N:(e + 1) * N], sw).t()
            continue
        w = _exact_blocks(s["qwt"][:, e * N:(e + 1) * N].t().contiguous(), sw)
        dy, f = s["dy"][a:b], s["dy_fmt"]
        y[a:b] = _exact_fp8(dy, f) @ w
        dw[e] = _exact_fp8(dy.t(), f) @ _exact_fp8(x.t()).t()
    return y if dw is None else (y, dw.view(E * N, K))
