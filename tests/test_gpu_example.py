"""The mixture-of-experts example runs: its loss falls, its 4-bit layer stays near the FP8 one, and one FP8 training
step's gradients are those of the layer's formula."""

import os
import sys

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from oracle import mx
from parity import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_example():
    import moe_layer

    say("moe example")
    losses, off_by = moe_layer.main(steps=6, tokens=300)
    assert losses[-1] < losses[0] and all(0.0 < v < 1.0 for v in off_by)


@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_served_tokens_follow_the_formula(tokens):
    """serve() against the layer on the oracle's 4-bit operands in float64.  Both round h, a and y to BF16 and the
    activations to 4 bits; a BF16 rounding that falls the other way can move a 4-bit code by a step (up to 1/4 of its
    value), so the bound is on the norm: 2^-8 for the roundings of y and a few per cent for moved codes."""
    import moe_layer

    say("moe serve", tokens)
    layer = moe_layer.Layer("cuda", seed=7)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(tokens, moe_layer.HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    got = layer.serve(x, layer.quantize_experts()).double().cpu()
    token, gate, off = (v.cpu() for v in moe_layer.route(x, layer.router))
    E = moe_layer.EXPERTS

    def q(t):
        return torch.from_numpy(mx.mx_values(*mx.quant_mx_rows(t.float().cpu().numpy())))

    w1, w2 = q(layer.w1).view(E, -1, moe_layer.HIDDEN), q(layer.w2).view(E, moe_layer.HIDDEN, -1)
    xq = q(x)[token]
    want = torch.zeros(tokens, moe_layer.HIDDEN, dtype=torch.float64)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            h = (xq[a:b] @ w1[e].t()).to(torch.bfloat16)
            y = (q(moe_layer.swiglu(h)) @ w2[e].t()).to(torch.bfloat16)
            want.index_add_(0, token[a:b], y.double() * gate[a:b].double())
    rel = float((got - want).norm() / want.norm())
    say("relative difference", rel)
    assert rel < 0.05


def test_step_gradients_follow_the_formula(monkeypatch):
    import moe_layer

    say("moe example gradients")
    layer = moe_layer.Layer("cuda", seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(300, moe_layer.HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn(300, moe_layer.HIDDEN, generator=g, device="cuda")
    grads = {}
    monkeypatch.setattr(fq, "hyperball_step_batch", lambda w, dw, **k: grads.update(dw1=dw[0], dw2=dw[1]))
    layer.step(x, target)
    # float32 autograd of the same layer
    token, gate, off = moe_layer.route(x, layer.router)
    w1 = layer.w1.clone().requires_grad_(True)
    w2 = layer.w2.clone().requires_grad_(True)
    out = torch.zeros(300, moe_layer.HIDDEN, device="cuda")
    parts = []
    for e in range(moe_layer.EXPERTS):
        a, b = int(off[e]), int(off[e + 1])
        h = x[token[a:b]].float() @ w1.view(moe_layer.EXPERTS, -1, moe_layer.HIDDEN)[e].t()
        gg, u = h.chunk(2, -1)
        parts.append((torch.nn.functional.silu(gg) * u) @ w2.view(moe_layer.EXPERTS, moe_layer.HIDDEN, -1)[e].t())
    out = out.index_add(0, token, torch.cat(parts) * gate)
    (out - target).square().mean().backward()
    for name, w in (("dw1", w1), ("dw2", w2)):
        rel = float((grads[name] - w.grad).norm() / w.grad.norm())
        say(name, rel)
        assert rel < 0.15  # E4M3 keeps 2^-4 of a value: a few roundings of about 3.6 % each, in square sum
