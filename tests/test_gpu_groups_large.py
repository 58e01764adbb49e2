"""Operands and outputs past 4 GiB in the grouped and MXFP4 entry points: the last expert's weights, the last rows of an
input and of an output lie beyond a 32-bit byte offset.  Codes are drawn directly (every byte of E2M1 pairs and the
finite E4M3 bytes are valid operands); the rows under test are checked in float64 on the device."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import synth
from parity import F32_ABS, say

pytestmark = pytest.mark.gpu
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def e4m3_codes(shape, seed):
    q = torch.randint(0, 0x7F, shape, dtype=torch.uint8, device="cuda", generator=gen(seed))
    q[..., ::2] |= 0x80
    return q


def check(got, a, b, what):
    y = a @ b.t()
    lim = F32_ABS * torch.outer(a.norm(dim=1), b.norm(dim=1)) * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
    assert bool(((got.double() - y).abs() <= lim).all()), what


def mx_values(q, s):
    lut = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=q.device)
    v = torch.stack([lut[(q & 15).long()], lut[(q >> 4).long()]], -1).flatten(1)
    sc = torch.exp2(s.permute(1, 0, 2).flatten(1).double() - 127)[:, :v.shape[1] // 32]
    return v * sc.repeat_interleave(32, 1)


def two_experts(E, T):
    """Offsets that put the tokens on the first and the last expert."""
    off = torch.full((E + 1,), T // 3, dtype=torch.int64)
    off[0], off[E] = 0, T
    return off.cuda()


def test_stacked_fp8_weights():
    E, N, K, T = 33, 65536, 2048, 40
    say("large grouped fprop / dgrad")
    x = synth.device_normal_bf16((T, K), 1, "cuda")
    off = two_experts(E, T)
    sw = torch.rand(E * N // 128, K // 128, device="cuda", generator=gen(2)) + 0.5
    qx, sx = fq.quantize_act_1x128(x)
    qw = e4m3_codes((E * N, K), 3)
    y = fq.grouped_gemm_fprop(qx, sx, off, qw, sw)
    xd = qx.view(torch.float8_e4m3fn).double() * sx.t().double().repeat_interleave(128, 1)
    for e, rows in ((0, slice(0, T // 3)), (E - 1, slice(T // 3, T))):
        for n0 in (0, N - 256):
            r0 = e * N + n0
            w = qw[r0:r0 + 256].view(torch.float8_e4m3fn).double()
            w = w * sw[r0 // 128:r0 // 128 + 2].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            check(y[rows, n0:n0 + 256], xd[rows], w, ("fprop", e, n0))
    del qw, y
    # dgrad over the last expert's window of W^T [K, E N]; contraction over N
    K2, N2 = 2048, 65536
    qwt = e4m3_codes((K2, E * N2), 4)
    sw = torch.rand(E * N2 // 128, K2 // 128, device="cuda", generator=gen(5)) + 0.5
    dy = synth.device_normal_bf16((T, N2), 6, "cuda", 1e-3)
    qd, sd = fq.quantize_act_1x128(dy)
    dx = fq.grouped_gemm_dgrad(qd, sd, off, qwt, sw)
    dd = qd.view(torch.float8_e4m3fn).double() * sd.t().double().repeat_interleave(128, 1)
    for e, rows in ((0, slice(0, T // 3)), (E - 1, slice(T // 3, T))):
        w = qwt[K2 - 128:, e * N2:(e + 1) * N2].view(torch.float8_e4m3fn).double()
        w = w * sw[e * N2 // 128:(e + 1) * N2 // 128, -1].double().repeat_interleave(128)
        check(dx[rows, K2 - 128:], dd[rows], w, ("dgrad", e))


def test_stacked_weight_gradient():
    E, N, K, T = 33, 32768, 2048, 200
    say("large grouped wgrad")
    off = two_experts(E, T)
    x, dy = synth.device_normal_bf16((T, K), 11, "cuda"), synth.device_normal_bf16((T, N), 12, "cuda", 1e-3)
    qxt, sxt = fq.quantize_act_grouped_128x1(x, off)
    qdt, sdt = fq.quantize_act_grouped_128x1(dy, off)
    dw = torch.full((E * N, K), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.grouped_gemm_wgrad(qdt, sdt, qxt, sxt, off, out=dw)
    for e in range(1, E - 1):
        assert not dw[e * N:(e + 1) * N].any(), e
    first = (T // 3 + 127) // 128
    for e, b0, b1 in ((0, 0, first), (E - 1, first, first + (T - T // 3 + 127) // 128)):
        xv = qxt[:, 128 * b0:128 * b1].view(torch.float8_e4m3fn).double() * sxt[b0:b1].t().double().repeat_interleave(128, 1)
        dv = qdt[-256:, 128 * b0:128 * b1].view(torch.float8_e4m3fn).double()
        dv = dv * sdt[b0:b1, -256:].t().double().repeat_interleave(128, 1)
        check(dw[e * N + N - 256:e * N + N], dv, xv, ("wgrad", e))


@pytest.mark.parametrize("T", [5, 40])
def test_stacked_4bit_weights(T):
    E, N, K = 65, 65536, 2048
    say("large grouped mx", T)
    g = gen(21)
    qw = torch.randint(0, 256, (E * N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    sw = torch.randint(110, 125, (K // 128, E * N, 4), dtype=torch.uint8, device="cuda", generator=g)
    x = synth.device_normal_bf16((T, K), 22, "cuda")
    off = two_experts(E, T)
    y = fq.grouped_linear_mxfp4(x, off, qw, sw)
    q, s = fq.quantize_mxfp4(x)
    xv = mx_values(q, s)
    for e, rows in ((0, slice(0, T // 3)), (E - 1, slice(T // 3, T))):
        for n0 in (0, N - 100):
            r = slice(e * N + n0, e * N + n0 + 100)
            check(y[rows, n0:n0 + 100], xv[rows], mx_values(qw[r], sw[:, r]), (e, n0))


def test_large_output_and_input():
    M, N, K = 70000, 32768, 64
    say("large mx output")
    x, w = synth.device_normal_bf16((M, K), 31, "cuda"), synth.device_normal_bf16((N, K), 32, "cuda")
    q, s = fq.quantize_mxfp4(x)
    qw, sw = fq.quantize_mxfp4(w)
    y = fq.gemm_mxfp4(q, s, qw, sw)
    check(y[-300:, -200:], mx_values(q[-300:], s[:, -300:]), mx_values(qw[-200:], sw[:, -200:]), "last corner")
    check(y[:64, :64], mx_values(q[:64], s[:, :64]), mx_values(qw[:64], sw[:, :64]), "first corner")
    # the output as an input past 4 GiB: its last rows and columns quantize as on their own
    qy, sy, qyt, syt = fq.quantize_mxfp4_dual(y)
    qe, se = fq.quantize_mxfp4(y[-300:].contiguous())
    assert torch.equal(qy[-300:], qe) and torch.equal(sy[:, -300:], se)
    r0 = (M - 300) // 128 * 128
    qe, se = fq.quantize_mxfp4_t(y[r0:, -64:].contiguous())
    assert torch.equal(qyt[-64:, r0 // 2:], qe) and torch.equal(syt[r0 // 128:, -64:], se)
