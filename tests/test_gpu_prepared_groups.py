"""prepare() on the grouped and MXFP4 entry points: the prepared launches give what the calls give, again and again, and see
new contents of the same buffers, new offsets among them."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import synth
from parity import say

pytestmark = pytest.mark.gpu


def test_prepared_calls():
    say("prepared grouped and mx")
    E, T, N, K = 4, 300, 256, 384
    u8 = dict(dtype=torch.uint8, device="cuda")
    x, dy = torch.empty(T, K, dtype=torch.bfloat16, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    w = synth.random_bf16((E * N, K), 800, 0.02).cuda()
    qw, sw, qwt = fq.quantize_weight_dual(w, fq.E4M3)
    q4, s4 = fq.quantize_mxfp4(w)
    p = fq.fp8bq_grouped_padded_rows(T, E)

    def quantized(C):
        return (torch.empty(T, C, **u8), torch.empty(C // 128, T, device="cuda"), torch.empty(C, p, **u8),
                torch.empty(p // 128, C, device="cuda"))

    (q, s, qt, st), (qd, sd, qdt, sdt) = quantized(K), quantized(N)
    y, dx = torch.empty(T, N, device="cuda"), torch.empty(T, K, device="cuda")
    dw = torch.empty(E * N, K, device="cuda")
    m, g = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    xq, xs = torch.empty(T, K // 2, **u8), torch.empty(3, T, 4, **u8)
    d, e, one = torch.empty(T, E * N, device="cuda"), torch.empty(T, E * N, device="cuda"), torch.empty(1, E * N, device="cuda")
    ws = torch.empty(max(fq.fp8bq_linear_mxfp4_workspace_size(T, E * N, K),
                         fq.fp8bq_grouped_linear_mxfp4_workspace_size(E, T, N, K),
                         fq.fp8bq_gemm_mxfp4_workspace_size(T, E * N, K), 16), **u8)
    f = fq.E4M3
    calls = [(fq.fp8bq_quantize_act_grouped, x, off, f, q, s, f, qt, st),
             (fq.fp8bq_quantize_act_grouped, dy, off, f, qd, sd, f, qdt, sdt),
             (fq.fp8bq_grouped_gemm_fprop, q, s, f, off, qw, sw, f, y),
             (fq.fp8bq_grouped_gemm_dgrad, qd, sd, f, off, qwt, sw, f, dx),
             (fq.fp8bq_grouped_gemm_wgrad, qdt, sdt, f, qt, st, f, off, dw),
             (fq.fp8bq_quantize_mxfp4, x, xq, xs, None, None),
             (fq.fp8bq_grouped_gemm_mxfp4, xq, xs, off, q4, s4, m),
             (fq.fp8bq_grouped_linear_mxfp4, x, off, q4, s4, g, ws),
             (fq.fp8bq_gemm_mxfp4, xq, xs, q4, s4, d, ws),
             (fq.fp8bq_linear_mxfp4, x, q4, s4, e, ws),
             (fq.fp8bq_linear_mxfp4, x[:1], q4, s4, one)]
    outs = (y, dx, dw, m, g, d, e, one)
    launches = [fq.prepare(*c) for c in calls]
    for i, cuts in enumerate(([0, 5, 5, 200, T], [0, 100, 101, 299, T], [0, T, T, T, T])):
        x.copy_(synth.random_bf16((T, K), 810 + i))
        dy.copy_(synth.random_bf16((T, N), 820 + i, 1e-3))
        off.copy_(torch.from_numpy(np.array(cuts, np.int64)))
        for launch in launches:
            launch()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.fill_(7.0)
        for fn, *args in calls:
            fn(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
        assert torch.equal(m, g) and torch.equal(d, e) and not torch.any(y == 7.0)
