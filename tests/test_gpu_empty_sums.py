"""Sums and maxima over nothing: rows of no elements have the dot product zero, and the smallest scale."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu


def soil(n):
    """Leaves numbers behind in the memory that the next allocations are made from."""
    for _ in range(4):
        torch.full((n,), 7.0, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_gradient_of_rows_without_elements(dtype):
    say("empty sums, combine backward", dtype)
    T, k = 37, 3
    experts = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) % 5
    _, rows, slots = fq.expert_rows(experts, 5)
    weights = torch.ones(T, k, device="cuda")
    soil(T * k)
    dy, dw = fq.combine_rows_backward(torch.zeros(T, 0, device="cuda"), torch.zeros(T * k, 0, device="cuda", dtype=dtype), rows,
                                      weights, slots)
    assert dy.shape == (T * k, 0) and dw.shape == (T, k) and not dw.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scales_of_rows_and_columns_without_elements(dtype):
    say("empty sums, 8-bit scales", dtype)
    least = torch.tensor(1e-12, device="cuda")
    soil(48)
    q, s = fq.quantize_int8(torch.zeros(48, 0, device="cuda", dtype=dtype))
    assert q.shape == (48, 0) and s.shape == (48,) and bool((s == least).all())
    soil(48)
    qt, st = fq.quantize_int8_t(torch.zeros(0, 48, device="cuda", dtype=dtype))
    assert qt.shape == (48, 0) and st.shape == (48,) and bool((st == least).all())
    y = fq.gemm_int8(q, s, qt, st)
    assert y.shape == (48, 48) and not y.any()
