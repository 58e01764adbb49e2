"""MXFP4 quantization of blocks near the smallest scales: the largest magnitude between 2^-133 and 2^-120, members down to
the smallest subnormals.  A block's scale is 2^-127 up to an amax below 2^-124 and doubles with every binade from there,
so members below 2^-126 (subnormal in BF16 and FP32) still have non-zero codes under the next three scales.  Codes and
scales bit for bit; the linear layer that quantizes its input itself against the float64 product of the oracle's
values, within 1e-4 ||a|| ||b|| (the FP32 rule of parity.py)."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import synth
from oracle import mx
from parity import F32_ABS, say, to_np_f64

pytestmark = pytest.mark.gpu


def tiny(R, C, dtype, seed):
    """Row r's blocks of 32 have amax in [2^a, 2^(a+1)), a = -133 + r % 14; the other members are spread over the
    binades below, signs both ways, some zeros."""
    rng = np.random.default_rng(seed)
    top = -133 + np.arange(R) % 14
    ex = top[:, None] - rng.integers(0, 8, (R, C))
    lead = rng.integers(0, 32, (R, C // 32)) + 32 * np.arange(C // 32)
    np.put_along_axis(ex, lead, top[:, None], 1)
    v = np.ldexp(1.0 + rng.integers(0, 128, (R, C)) / 128.0, ex) * rng.choice([-1.0, 1.0], (R, C))
    v[rng.random((R, C)) < 0.05] = -0.0
    return torch.from_numpy(v.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(28, 64), (140, 160), (256, 256)])
def test_codes_and_scales(R, C, dtype):
    say("mx small blocks", R, C, dtype)
    x = tiny(R, C, dtype, R + C)
    code, scale = mx.quant_mx_rows(x.float().numpy())
    assert {0, 1, 2, 3} <= set(np.unique(scale))
    q, s = fq.quantize_mxfp4(x.cuda())
    qd, sd, _, _ = fq.quantize_mxfp4_dual(x.cuda())
    n = R // 8 * 8  # (a column quantizer's width is a multiple of 8)
    qt, st = fq.quantize_mxfp4_t(x[:n].t().contiguous().cuda())  # the same blocks down the columns
    torch.cuda.synchronize()
    for got_q, got_s, r in ((q, s, R), (qd, sd, R), (qt, st, n)):
        assert np.array_equal(got_s.cpu().numpy(), mx.scale_words(scale[:r]))
        assert np.array_equal(got_q.cpu().numpy(), mx.pack(code[:r]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 14, 16, 56])
def test_linear_quantizes_them_alike(M, dtype):
    say("mx small blocks linear", M, dtype)
    N, K = 48, 256
    x = tiny(16, K, dtype, 5)[:M] if M <= 16 else tiny(M, K, dtype, 6)
    if M == 1:
        x = tiny(16, K, dtype, 7)[9:10]  # amax about 2^-124
    w = synth.random_bf16((N, K), 8, 1.0).float().numpy() * np.float32(2.0 ** 100)
    code, scale = mx.quant_mx_rows(w)
    y = fq.linear_mxfp4(x.cuda(), torch.from_numpy(mx.pack(code)).cuda(), torch.from_numpy(mx.scale_words(scale)).cuda(),
                        out_dtype=torch.float32)
    off = torch.tensor([0, M // 2, M], device="cuda")
    yg = fq.grouped_linear_mxfp4(x.cuda(), off, torch.from_numpy(mx.pack(np.concatenate([code, code]))).cuda(),
                                 torch.from_numpy(mx.scale_words(np.concatenate([scale, scale]))).cuda(),
                                 out_dtype=torch.float32)
    a, b = mx.mx_values(*mx.quant_mx_rows(x.float().numpy())), mx.mx_values(code, scale)
    lim = F32_ABS * np.outer(np.linalg.norm(a, axis=1), np.linalg.norm(b, axis=1))
    for got in (y, yg):
        assert np.all(np.abs(to_np_f64(got) - a @ b.T) <= lim)
