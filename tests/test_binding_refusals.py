"""What the bindings of the grouped and MXFP4 entry points refuse before any launch, without a GPU: arguments that are
no tensors, missing ones, and offsets that name no expert are told by name, with the exception type of the other
arguments."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq

E, T, N, K = 4, 300, 256, 384
TP = 768


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s)


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


OFF = torch.zeros(E + 1, dtype=torch.int64)
CALLS = {  # entry point: (arguments, positions of those that may be None)
    "fp8bq_quantize_act_grouped": ([bf16(T, K), OFF, 0, u8(T, K), f32(K // 128, T), 0, u8(K, TP), f32(TP // 128, K)], {3, 4}),
    "fp8bq_grouped_gemm_fprop": ([u8(T, K), f32(K // 128, T), 0, OFF, u8(E * N, K), f32(E * N // 128, K // 128), 0,
                                  bf16(T, N)], set()),
    "fp8bq_grouped_gemm_dgrad": ([u8(T, N), f32(N // 128, T), 0, OFF, u8(K, E * N), f32(E * N // 128, K // 128), 0,
                                  bf16(T, K)], set()),
    "fp8bq_grouped_gemm_wgrad": ([u8(N, TP), f32(TP // 128, N), 0, u8(K, TP), f32(TP // 128, K), 0, OFF, bf16(E * N, K)],
                                 set()),
    "fp8bq_quantize_mxfp4": ([bf16(T, K), u8(T, K // 2), u8(3, T, 4), u8(K, 160), u8(3, K, 4)], {1, 2, 3, 4}),
    "fp8bq_gemm_mxfp4": ([u8(T, K // 2), u8(3, T, 4), u8(N, K // 2), u8(3, N, 4), bf16(T, N)], set()),
    "fp8bq_linear_mxfp4": ([bf16(T, K), u8(N, K // 2), u8(3, N, 4), bf16(T, N)], set()),
    "fp8bq_grouped_gemm_mxfp4": ([u8(T, K // 2), u8(3, T, 4), OFF, u8(E * N, K // 2), u8(3, E * N, 4), bf16(T, N)], set()),
    "fp8bq_grouped_linear_mxfp4": ([bf16(T, K), OFF, u8(E * N, K // 2), u8(3, E * N, 4), bf16(T, N)], set()),
}
# every tensor argument but the one the sizes come from and weights, whose rows are counted first
PLACES = [(name, i) for name, (args, _) in sorted(CALLS.items()) for i, a in enumerate(args)
          if i > 0 and isinstance(a, torch.Tensor) and not (a.dim() == 2 and a.dtype == torch.uint8 and a.shape[0] in (N, E * N, K)
                                                            and name != "fp8bq_quantize_act_grouped")]


@pytest.mark.parametrize("name,place", PLACES)
def test_missing_tensors_and_other_objects(name, place):
    args, optional = CALLS[name]
    for bad in ([1, 2], 5) if place in optional else (None, [1, 2], 5):
        call = list(args)
        call[place] = bad
        with pytest.raises(TypeError):
            getattr(fq, name)(*call)


def test_offsets_that_name_no_expert():
    x = bf16(T, K)
    helpers = (lambda o: fq.quantize_act_grouped_128x1(x, o), lambda o: fq.quantize_act_grouped_dual(x, o),
               lambda o: fq.grouped_gemm_fprop(u8(T, K), f32(3, T), o, u8(E * N, K), f32(E * 2, 3)),
               lambda o: fq.grouped_gemm_dgrad(u8(T, N), f32(2, T), o, u8(K, E * N), f32(E * 2, 3)),
               lambda o: fq.grouped_gemm_wgrad(u8(N, TP), f32(6, N), u8(K, TP), f32(6, K), o),
               lambda o: fq.grouped_gemm_mxfp4(u8(T, K // 2), u8(3, T, 4), o, u8(E * N, K // 2), u8(3, E * N, 4)),
               lambda o: fq.grouped_linear_mxfp4(x, o, u8(E * N, K // 2), u8(3, E * N, 4)))
    for helper in helpers:
        for bad in (OFF[:1], OFF[:0], OFF[0]):
            with pytest.raises(ValueError):
                helper(bad)
        with pytest.raises(TypeError):
            helper([0, T])
