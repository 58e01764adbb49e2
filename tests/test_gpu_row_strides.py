"""Rows of the experts whose leading dimensions are not their width: the same values as with contiguous matrices (which are held
to float64 elsewhere), and nothing written between the rows."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def apart(t, gap, fill=0.0):
    """t's values in a matrix whose rows lie gap elements further apart, with gap values of `fill` behind each."""
    big = torch.full((t.shape[0], t.shape[1] + gap), fill, dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big, big[:, :t.shape[1]]


def case(T, k, H, E, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    experts = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    experts[torch.rand(T, k, generator=g, device="cuda") < 0.2] = -1
    _, rows, slots = fq.expert_rows(experts.contiguous(), E)
    w = torch.rand(T, k, generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    y = torch.randn(T * k, H, generator=g, device="cuda").to(dtype)
    return rows, slots, w, x, y


@pytest.mark.parametrize("T,k,H,E", [(1, 1, 8, 1), (37, 3, 264, 7), (300, 2, 2048, 16), (65, 6, 4104, 9)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gap", [8, 24, 1000])
def test_moves(T, k, H, E, dtype, gap):
    say("row strides", T, k, H, dtype, gap)
    rows, slots, w, x, y = case(T, k, H, E, dtype)
    n = T * k
    want = fq.gather_rows(x, slots, k)
    big, out = apart(torch.zeros_like(want), gap, 7.0)
    fq.fp8bq_gather_rows(apart(x, 2 * gap)[1], slots, k, out)
    assert torch.equal(out, want) and bool((big[:, H:] == 7.0).all())
    for out_dtype in (BF16, F32):
        for weights in (w, None):
            want = fq.combine_rows(y, rows, weights, out_dtype=out_dtype)
            big, out = apart(torch.zeros_like(want), gap, 7.0)
            fq.fp8bq_combine_rows(apart(y, 3 * gap, float("nan"))[1], rows, weights, out)
            assert torch.equal(out, want) and bool((big[:, H:] == 7.0).all())
        dout = x.to(out_dtype)
        dy, dw = fq.combine_rows_backward(dout, y, rows, w, slots)
        big, got = apart(torch.ones(n, H, dtype=dtype, device="cuda"), gap, 7.0)
        gotw = torch.full_like(w, 9.0)
        fq.fp8bq_combine_rows_backward(apart(dout, gap, float("nan"))[1], apart(y, 2 * gap, float("nan"))[1], rows, w, slots, got,
                                       gotw)
        assert torch.equal(got, dy) and torch.equal(gotw, dw) and bool((big[:, H:] == 7.0).all())


def test_plain_values():
    """The strided forms against float64: sums of three products, each off by half a step of FP32 a factor and a sum, and one
    rounding of the result."""
    say("row strides, float64")
    T, k, H, E = 61, 3, 136, 5
    rows, slots, w, x, y = case(T, k, H, E, F32)
    yd, held = y.double()[rows.clamp(min=0).long()], (rows >= 0).unsqueeze(-1)
    yd = torch.where(held, yd, 0.0)
    out = torch.empty(T, H + 8, device="cuda")[:, :H]
    fq.fp8bq_combine_rows(apart(y, 8)[1], rows, w, out)
    terms = yd * w.double().unsqueeze(-1)
    assert bool(((out.double() - terms.sum(1)).abs() <= 4 * 2.0 ** -24 * terms.abs().sum(1)).all())
    dy, dw = torch.empty(T * k, H + 16, device="cuda")[:, :H], torch.empty(T, k, device="cuda")
    fq.fp8bq_combine_rows_backward(apart(x, 8)[1], apart(y, 8)[1], rows, w, slots, dy, dw)
    terms = yd * x.double().unsqueeze(1)
    # 136 products: a lane adds eight of them, then six levels of lanes and three of waves: 17 roundings
    assert bool(((dw.double() - terms.sum(-1)).abs() <= 18 * 2.0 ** -24 * terms.abs().sum(-1)).all())
    want = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    mine = rows.flatten() >= 0
    want[rows.flatten()[mine].long()] = (x.double().unsqueeze(1) * w.double().unsqueeze(-1)).view(T * k, H)[mine]
    assert bool(((dy.double() - want).abs() <= 2.0 ** -24 * want.abs()).all())
