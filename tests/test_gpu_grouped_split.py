"""Weight gradients of unevenly loaded experts, whose long contractions are split over workgroups and added up in FP32:
against the float64 product of the same codes, within 1e-4 ||a|| ||b|| (FP32 sums in blocks of 128 tokens, in
whatever order) and for a BF16 output half a unit in its last place more, 2^-8 |y|."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_amd as fq
import synth
from parity import F32_ABS, say

pytestmark = pytest.mark.gpu

# (tokens of each expert, N, K): one expert with nearly everything, two long ones, everything on one of many, all even and
# few tiles, a last block with one token, more experts than a wave has lanes
CASES = {
    "one_long": ([7003, 0, 130, 1], 256, 128),
    "two_long": ([40, 4000, 300, 3900, 0, 1, 77, 128], 128, 384),
    "all_on_one": ([0, 0, 8193, 0, 0], 384, 256),
    "one_expert": ([20001], 256, 256),
    "even": ([2300] * 4, 128, 128),
    "many_experts": ([9 if e % 3 else 0 for e in range(200)] + [6000], 128, 128),
    "wide": ([9000, 500, 0, 3], 1408, 512),
}


def operands(counts, N, K, seed):
    T, E = sum(counts), len(counts)
    x = synth.random_bf16((T, K), seed, 1.0, outliers=True).cuda()
    dy = synth.random_bf16((T, N), seed + 1, 1e-3).cuda()
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)).cuda()
    return off, fq.quantize_act_grouped_128x1(dy, off, fq.E5M2), fq.quantize_act_grouped_128x1(x, off)


def expected(counts, qdyt, sdyt, qxt, sxt):
    """(dW, bound without the output's rounding) of every expert in float64."""
    ys, lims, p = [], [], 0
    for n in counts:
        b = (n + 127) // 128
        part = []
        for q, s, t in ((qdyt, sdyt, torch.float8_e5m2), (qxt, sxt, torch.float8_e4m3fn)):
            v = q[:, p:p + 128 * b].contiguous().view(t).double()
            part.append(v * s[p // 128:p // 128 + b].double().t().repeat_interleave(128, 1))
        p += 128 * b
        a, c = part
        ys.append(a @ c.t().contiguous())
        lims.append(F32_ABS * torch.outer(a.norm(dim=1), c.norm(dim=1)))
    return torch.cat(ys), torch.cat(lims)


@pytest.mark.parametrize("name", sorted(CASES))
def test_split_experts(name):
    say("grouped split", name)
    counts, N, K = CASES[name]
    E = len(counts)
    off, (qdyt, sdyt), (qxt, sxt) = operands(counts, N, K, 300)
    size = fq.fp8bq_grouped_gemm_wgrad_workspace_size(E, qdyt.shape[1], N, K)
    assert size > 0
    y, lim = expected(counts, qdyt, sdyt, qxt, sxt)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # (NaNs, and a guard behind)
    for dtype in (torch.bfloat16, torch.float32):
        for space in (ws[:size], None):
            big = torch.full((E * N + 2, K + 16), 7.0, dtype=dtype, device="cuda")
            dw = big[1:-1, :K] if dtype == torch.float32 else big[:-2, :K]
            fq.fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fq.E5M2, qxt, sxt, fq.E4M3, off, dw, ws=space)
            torch.cuda.synchronize()
            bound = lim if dtype == torch.float32 else lim * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
            assert torch.all((dw.double() - y).abs() <= bound), (dtype, space is None)
            dw.fill_(7.0)
            assert torch.all(big == 7.0)
    assert torch.all(ws[size:] == 0xFF)
    one = fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, off, fq.E5M2, out_dtype=torch.float32)
    again = fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, off, fq.E5M2, out_dtype=torch.float32)
    start = torch.randn(E * N, K, device="cuda")
    acc = start.clone()
    fq.grouped_gemm_wgrad(qdyt, sdyt, qxt, sxt, off, fq.E5M2, out=acc, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(one, again) and torch.equal(acc, start + one)


def test_new_offsets_in_a_graph():
    """A captured product follows the counts it finds on the device: split, then not, then split elsewhere."""
    say("grouped split graph")
    N = K = 128
    E, T = 4, 8000
    x = synth.random_bf16((T, K), 400, 1.0).cuda()
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    loads = [[8000, 0, 0, 0], [2000] * 4, [1, 7, 7900, 92], [0, 0, 0, 0]]

    def fill(counts):
        off.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)))

    def step():
        qt, st = fq.quantize_act_grouped_128x1(x, off)
        return qt, st, fq.grouped_gemm_wgrad(qt, st, qt, st, off, out_dtype=torch.float32)

    fill(loads[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qt, st, dw = step()
    for counts in loads + loads[:2]:
        fill(counts)
        graph.replay()
        torch.cuda.synchronize()
        got = dw.clone()
        eager = step()[2]
        torch.cuda.synchronize()
        assert torch.equal(got, eager), counts
        p = 0
        for e, n in enumerate(counts):
            b = (n + 127) // 128
            v = qt[:, p:p + 128 * b].contiguous().view(torch.float8_e4m3fn).double()
            v = v * st[p // 128:p // 128 + b].double().t().repeat_interleave(128, 1)
            p += 128 * b
            y, m = v @ v.t().contiguous(), v.norm(dim=1)
            assert torch.all((got[e * N:(e + 1) * N].double() - y).abs() <= F32_ABS * torch.outer(m, m)), (counts, e)
