"""A mixture-of-experts feed-forward layer: trained in FP8, served with its experts in 4 or 8 bits.

    python examples/moe_layer.py

Each token goes to its top two of eight experts; an expert is SwiGLU, y = W2 (silu(g) * u) with (g, u) = W1 x.
The training step routes, brings the rows to their experts and back, runs the grouped FP8 products forward and backward
(token counts stay on the device) and updates the FP32 master weights with the batched Hyperball step, along the
gradients or, as MuonH does, along their orthogonalized form; it may train the router too.  Then the experts are
quantized to MXFP4 or to 8-bit integers and single tokens are served through the grouped linear layers.  Prints the
loss of a few steps towards another such layer's output and how far the 4- and 8-bit layers are from the FP8 one (each
of the 4-bit layer's two products rounds both operands to a digit or so).
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_blockwise_quantized_amd as fq  # noqa: E402

HIDDEN, FFN, EXPERTS, TOP = 512, 384, 8, 2


def choose(x, router):
    """The router's logits, each token's experts and weights, and where its rows lie among the experts' rows."""
    logits = x.float() @ router
    experts, gate = fq.route_experts(logits, TOP)
    return (logits, experts, gate) + fq.expert_rows(experts, EXPERTS)


def route(x, router):
    """Rows sorted by expert: (token of each row, its weight, offsets [E + 1]), all on the device."""
    _, _, gate, offsets, _, slots = choose(x, router)
    return slots.long() // TOP, gate.flatten()[slots.long()].unsqueeze(1), offsets


def swiglu(h):
    g, u = h.float().chunk(2, -1)
    return (torch.nn.functional.silu(g) * u).to(torch.bfloat16)


def swiglu_backward(h, da):
    g, u = h.float().chunk(2, -1)
    s = torch.sigmoid(g)
    da = da.float()
    return torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], -1).to(torch.bfloat16)


class Layer:
    """Master weights in FP32, stacked by expert: w1 [E 2 FFN, HIDDEN], w2 [E HIDDEN, FFN]."""

    def __init__(self, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.w1 = torch.randn(EXPERTS * 2 * FFN, HIDDEN, generator=g, device=device) * HIDDEN ** -0.5
        self.w2 = torch.randn(EXPERTS * HIDDEN, FFN, generator=g, device=device) * FFN ** -0.5
        self.router = torch.randn(HIDDEN, EXPERTS, generator=g, device=device) * HIDDEN ** -0.5

    def step(self, x, target, lr=0.02, orthogonal=False, router_lr=0.0):
        """One training step on the experts' weights, and with router_lr on the router's; returns the mean squared error
        before it.  orthogonal: along the orthogonalized gradient of each expert's matrices."""
        logits, experts, gate, off, rows_of, slots = choose(x, self.router)
        (q1, s1, q1t), (q2, s2, q2t) = fq.quantize_weights_dual([self.w1, self.w2])
        # forward
        rows = fq.gather_rows(x, slots, TOP)
        qx, sx, qxt, sxt = fq.quantize_act_grouped_dual(rows, off)
        h = fq.grouped_gemm_fprop(qx, sx, off, q1, s1)
        a = swiglu(h)
        qa, sa, qat, sat = fq.quantize_act_grouped_dual(a, off)
        y = fq.grouped_gemm_fprop(qa, sa, off, q2, s2)
        out = fq.combine_rows(y, rows_of, gate, out_dtype=torch.float32)
        loss = (out - target).square().mean()
        # backward
        dout = (2.0 / out.numel()) * (out - target)
        dy, dgate = fq.combine_rows_backward(dout, y, rows_of, gate, slots)
        qd, sd, qdt, sdt = fq.quantize_act_grouped_dual(dy, off)
        da = fq.grouped_gemm_dgrad(qd, sd, off, q2t, s2)
        dw2 = fq.grouped_gemm_wgrad(qdt, sdt, qat, sat, off, out_dtype=torch.float32)
        dh = swiglu_backward(h, da)
        dw1 = fq.grouped_gemm_wgrad(*fq.quantize_act_grouped_128x1(dh, off), qxt, sxt, off, out_dtype=torch.float32)
        if orthogonal:  # (an expert without tokens has a zero gradient, and keeps it)
            dw1, dw2 = (fq.orthogonalize(d.view(EXPERTS, -1, d.shape[1])).view(d.shape) for d in (dw1, dw2))
        fq.hyperball_step_batch([self.w1, self.w2], [dw1, dw2], lr=lr * self.w1.norm().item(), weight_decay=0.0)
        if router_lr:
            self.router -= router_lr * (x.float().t() @ fq.route_experts_backward(dgate, logits, experts))
        return float(loss)

    def forward_fp8(self, x):
        _, _, gate, off, rows_of, slots = choose(x, self.router)
        (q1, s1, _), (q2, s2, _) = fq.quantize_weights_dual([self.w1, self.w2])
        h = fq.grouped_gemm_fprop(*fq.quantize_act_1x128(fq.gather_rows(x, slots, TOP)), off, q1, s1)
        y = fq.grouped_gemm_fprop(*fq.quantize_act_1x128(swiglu(h)), off, q2, s2)
        return fq.combine_rows(y, rows_of, gate, out_dtype=torch.float32)

    def quantize_experts(self):
        """The experts in 4 bits, laid out once for serving."""
        return fq.quantize_mxfp4(self.w1), fq.quantize_mxfp4(self.w2)

    def serve(self, x, experts):
        return self._serve(x, experts, fq.grouped_linear_mxfp4)

    def quantize_experts_int8(self):
        """The experts in 8 bits, a scale for each output channel."""
        return fq.quantize_int8(self.w1), fq.quantize_int8(self.w2)

    def serve_int8(self, x, experts):
        return self._serve(x, experts, fq.grouped_linear_int8)

    def _serve(self, x, experts, linear):
        (q1, s1), (q2, s2) = experts
        _, _, gate, off, rows_of, slots = choose(x, self.router)
        h = linear(fq.gather_rows(x, slots, TOP), off, q1, s1)
        y = linear(swiglu(h), off, q2, s2)
        return fq.combine_rows(y, rows_of, gate, out_dtype=torch.float32)


def main(steps=8, tokens=777, device="cuda"):
    g = torch.Generator(device=device).manual_seed(1)
    layer = Layer(device)
    x = torch.randn(tokens, HIDDEN, generator=g, device=device).to(torch.bfloat16)
    target = Layer(device, seed=2).forward_fp8(x)
    losses = [layer.step(x, target) for _ in range(steps)]
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    along = Layer(device)
    print("along orthogonalized gradients, router trained too",
          " ".join(f"{along.step(x, target, orthogonal=True, router_lr=10.0):.4f}" for _ in range(steps)))
    experts = layer.quantize_experts()
    exact = layer.forward_fp8(x)
    off_by = [float((layer.serve(x[:n], experts) - exact[:n]).norm() / exact[:n].norm()) for n in (1, 7, tokens)]
    eight = layer.quantize_experts_int8()
    off_by8 = [float((layer.serve_int8(x[:n], eight) - exact[:n]).norm() / exact[:n].norm()) for n in (1, 7, tokens)]
    print("8-bit layer against FP8, relative error for 1, 7 and %d tokens: %s" % (tokens, " ".join(f"{v:.3f}" for v in off_by8)))
    print("4-bit layer against FP8, relative error for 1, 7 and %d tokens: %s" % (tokens, " ".join(f"{v:.3f}" for v in off_by)))
    return losses, off_by


if __name__ == "__main__":
    main()
