"""The entry points and helpers of routing, the 8-bit layer and the orthogonalization take every argument by the name that
their signature shows, without a GPU: the call goes as far as the check of the device, which comes last."""

import inspect

import pytest
import torch

import fp8_blockwise_quantized_amd as fq

T, K, E, H, N = 6, 2, 4, 16, 8
X, CODES, CHOICES = torch.zeros(T, H), torch.zeros(N, H, dtype=torch.int8), torch.zeros(T, K, dtype=torch.int32)
SLOTS, WEIGHTS, TALL = torch.zeros(T * K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(T * K, H)
OFF = torch.zeros(E + 1, dtype=torch.int64)
LOGITS = torch.zeros(T, E)


def codes(r):
    return torch.zeros(r, H, dtype=torch.int8)


HELPERS = {
    "quantize_int8": dict(x=X),
    "quantize_int8_t": dict(x=X),
    "gemm_int8": dict(qa=codes(T), sa=torch.zeros(T), qb=CODES, sb=torch.zeros(N)),
    "linear_int8": dict(x=X, qw=CODES, sw=torch.zeros(N)),
    "grouped_gemm_int8": dict(qa=codes(T), sa=torch.zeros(T), offsets=OFF, qw=codes(E * N), sw=torch.zeros(E * N)),
    "grouped_linear_int8": dict(x=X, offsets=OFF, qw=codes(E * N), sw=torch.zeros(E * N)),
    "route_experts": dict(logits=LOGITS, k=K),
    "route_experts_backward": dict(dweights=WEIGHTS, logits=LOGITS, experts=CHOICES),
    "expert_rows": dict(experts=CHOICES, E=E),
    "gather_rows": dict(x=X, slots=SLOTS, k=K),
    "combine_rows": dict(y=TALL, rows=CHOICES, weights=WEIGHTS),
    "combine_rows_backward": dict(dout=X, y=TALL, rows=CHOICES, weights=WEIGHTS, slots=SLOTS),
    "orthogonalize": dict(g=X),
}
ENTRIES = {
    "fp8bq_quantize_int8": dict(x=X, q=codes(T), s=torch.zeros(T)),
    "fp8bq_linear_int8": dict(x=X, qw=CODES, sw=torch.zeros(N), y=torch.zeros(T, N)),
    "fp8bq_route_experts": dict(logits=LOGITS, k=K, score=0, bias=None, groups=1, top_groups=1, group_best=1, renormalize=True,
                                scale=1.0, experts=CHOICES, weights=WEIGHTS),
    "fp8bq_gather_rows": dict(x=X, slots=SLOTS, k=K, out=TALL),
    "fp8bq_orthogonalize": dict(g=X, coefficients=[(1.5, -0.5, 0.0)], eps=1e-7, out=X.bfloat16(), ws=None),
}
CALLS = {**HELPERS, **ENTRIES}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("turn", [False, True])
def test_all_by_name(name, turn):
    args = CALLS[name]
    with pytest.raises(ValueError, match="CUDA"):
        getattr(fq, name)(**dict(reversed(args.items())) if turn else args)


@pytest.mark.parametrize("name", sorted(HELPERS))
def test_the_names_are_those_of_the_signature(name):
    assert set(HELPERS[name]) <= set(inspect.signature(getattr(fq, name)).parameters)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_nothing_given(name):
    with pytest.raises(TypeError, match="missing"):
        getattr(fq, name)()
