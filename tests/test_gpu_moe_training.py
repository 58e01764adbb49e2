"""A mixture-of-experts layer's step as a training loop chains the operators: routing, rows, grouped FP8 products,
their gradients, the orthogonalized update and the normalized step; and the layer served in 8 bits."""

import os
import sys

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

F64 = torch.float64


def inputs(tokens, seed, scale=1.0):
    import moe_layer

    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(tokens, moe_layer.HIDDEN, generator=g, device="cuda") * scale).to(torch.bfloat16)
    return x, torch.randn(tokens, moe_layer.HIDDEN, generator=g, device="cuda")


def forward64(layer, x, router):
    """The layer's formula in 64 bits, differentiable in the router."""
    import moe_layer as m

    logits = x.to(F64) @ router
    experts = fq.route_experts(x.float() @ layer.router, m.TOP)[0].long()
    gate = torch.softmax(logits.gather(1, experts), 1)
    w1, w2 = layer.w1.to(F64).view(m.EXPERTS, -1, m.HIDDEN), layer.w2.to(F64).view(m.EXPERTS, m.HIDDEN, -1)
    out = torch.zeros(x.shape, dtype=F64, device="cuda")
    for e in range(m.EXPERTS):
        t, j = (experts == e).nonzero(as_tuple=True)
        g, u = (x[t].to(F64) @ w1[e].t()).chunk(2, -1)
        out = out.index_add(0, t, ((torch.nn.functional.silu(g) * u) @ w2[e].t()) * gate[t, j].unsqueeze(1))
    return out


@pytest.mark.parametrize("tokens", [1, 300])
def test_router_gradient_follows_the_formula(tokens):
    import moe_layer

    say("moe router gradient", tokens)
    layer = moe_layer.Layer("cuda", seed=3)
    x, target = inputs(tokens, 5)
    before = layer.router.clone()
    router = layer.router.to(F64).requires_grad_(True)
    (forward64(layer, x, router) - target).square().mean().backward()
    layer.step(x, target, router_lr=1.0)
    got = (before - layer.router).to(F64)
    # FP8 operands keep 2^-4 of a value: the experts' answers are off by about 5 %, in square sum over two products, and
    # with them the residual and the weights' gradients; the router's own step in FP32 adds 2^-24 of its weights
    rel = float((got - router.grad).norm() / router.grad.norm())
    say("relative", rel)
    assert rel < 0.15


def test_orthogonal_step():
    """The step along the orthogonalized gradients: the matrices move by lr along U V^T-like directions of each expert."""
    import moe_layer as m

    say("moe orthogonal step")
    x, target = inputs(300, 7)
    plain, along = m.Layer("cuda", seed=3), m.Layer("cuda", seed=3)
    seen = {}
    real = fq.hyperball_step_batch

    def watch(w, g, **k):
        seen["g"] = [t.clone() for t in g]
        return real(w, g, **k)

    fq.hyperball_step_batch = watch
    try:
        a = plain.step(x, target)
        raw = seen["g"]
        b = along.step(x, target, orthogonal=True)
        turned = seen["g"]
    finally:
        fq.hyperball_step_batch = real
    assert a == b
    for r, o in zip(raw, turned):
        E = m.EXPERTS
        assert torch.equal(o, fq.orthogonalize(r.view(E, -1, r.shape[1])).view(r.shape))
    for w0, w1 in zip((m.Layer("cuda", seed=3).w1,), (along.w1,)):
        moved = (w1 - w0).to(F64).norm()
        want = 0.02 * w0.norm().item()
        # FP32 weights: a move of that norm, each element rounded by 2^-24 of the weight
        assert abs(float(moved) - want) <= 2.0 ** -20 * want + 2.0 ** -24 * float(w0.to(F64).norm())


@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_served_in_8_bits(tokens):
    """serve_int8() against the layer on the 8-bit operands' values in float64: both round h, a and y to BF16, and a
    rounding of h or a that falls the other way moves an 8-bit code by one of up to 127."""
    import moe_layer as m

    say("moe serve 8 bits", tokens)
    layer = m.Layer("cuda", seed=7)
    x, _ = inputs(tokens, 9)
    got = layer.serve_int8(x, layer.quantize_experts_int8())
    token, gate, off = m.route(x, layer.router)

    def q(t):
        c, s = fq.quantize_int8(t.contiguous())
        return c.to(F64) * s.to(F64).unsqueeze(1)

    w1, w2 = q(layer.w1).view(m.EXPERTS, -1, m.HIDDEN), q(layer.w2).view(m.EXPERTS, m.HIDDEN, -1)
    want = torch.zeros(tokens, m.HIDDEN, dtype=F64, device="cuda")
    xq, o = q(x)[token], off.tolist()
    for e in range(m.EXPERTS):
        a, b = o[e], o[e + 1]
        if a < b:
            h = (xq[a:b] @ w1[e].t()).to(torch.bfloat16)
            y = (q(m.swiglu(h)) @ w2[e].t()).to(torch.bfloat16)
            want.index_add_(0, token[a:b], y.to(F64) * gate[a:b].to(F64))
    rel = float((got.to(F64) - want).norm() / want.norm())
    say("relative difference", rel)
    assert rel < 2.0 ** -8 + 1.0 / 127  # BF16 roundings that fall the other way, and a code that moves with one


def test_example_prints_and_steps():
    import moe_layer

    say("moe example, orthogonal")
    layer = moe_layer.Layer("cuda", seed=1)
    x, target = inputs(77, 3)
    losses = [layer.step(x, target, orthogonal=True, router_lr=1.0) for _ in range(3)]
    assert all(v == v and v < float("inf") for v in losses)
    assert bool(torch.isfinite(layer.router).all() and torch.isfinite(layer.w1).all() and torch.isfinite(layer.w2).all())
