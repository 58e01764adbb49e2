"""prepare() on the entry points of routing, the experts' rows, the 8-bit layer and the orthogonalization: the prepared launches
give what the calls give, again and again, on new values in the same tensors; and chains of them on two streams at once."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32


def new(*shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def space(n):
    return new(max(n, 16), dtype=torch.uint8)


class Chain:
    """Every entry point once, one behind the other, in tensors of its own."""

    def __init__(self, T=70, k=2, E=6, H=128, N=64, seed=1):
        self.sizes = T, k, E, H, N
        self.logits, self.x, self.w = new(T, E), new(T, H, dtype=BF16), new(E * N, H)
        self.fill(seed)
        ch, gate, off, rows, slots = new(T, k, dtype=I32), new(T, k), new(E + 1, dtype=torch.int64), new(T, k, dtype=I32), new(T * k, dtype=I32)
        xs, qx, sx = new(T * k, H, dtype=BF16), new(T * k, H, dtype=I8), new(T * k)
        qw, sw = new(E * N, H, dtype=I8), new(E * N)
        y, y2, out = new(T * k, N, dtype=BF16), new(T * k, N, dtype=BF16), new(T, N)
        dy, dgate, dlogits = new(T * k, N, dtype=BF16), new(T, k), new(T, E)
        padded = (T * k + 15) // 16 * 16
        qdt, sdt, qxt, sxt = new(N, padded, dtype=I8), new(N), new(H, padded, dtype=I8), new(H)
        dw, lin, o = new(N, H), new(T, N), new(E, N, H, dtype=BF16)
        n = T * k
        self.outputs = [ch, gate, off, rows, slots, xs, qx, sx, qw, sw, y, y2, out, dy, dgate, dlogits, qdt, sdt, qxt, sxt, dw, lin, o]
        self.calls = [
            (fq.fp8bq_route_experts, self.logits, k, 0, None, 1, 1, 1, True, 1.0, ch, gate),
            (fq.fp8bq_expert_rows, ch, E, off, rows, slots, space(fq.fp8bq_expert_rows_workspace_size(n, E))),
            (fq.fp8bq_gather_rows, self.x, slots, k, xs),
            (fq.fp8bq_quantize_int8, xs, qx, sx),
            (fq.fp8bq_quantize_int8, self.w, qw, sw),
            (fq.fp8bq_grouped_gemm_int8, qx, sx, off, qw, sw, y, space(fq.fp8bq_grouped_gemm_int8_workspace_size(E, n, N, H))),
            (fq.fp8bq_grouped_linear_int8, xs, off, qw, sw, y2, space(fq.fp8bq_grouped_linear_int8_workspace_size(E, n, N, H))),
            (fq.fp8bq_combine_rows, y, rows, gate, out),
            (fq.fp8bq_combine_rows_backward, out, y, rows, gate, slots, dy, dgate),
            (fq.fp8bq_route_experts_backward, dgate, self.logits, 0, True, 1.0, ch, dlogits),
            (fq.fp8bq_quantize_int8_t, dy, qdt, sdt, space(fq.fp8bq_quantize_int8_t_workspace_size(n, N))),
            (fq.fp8bq_quantize_int8_t, xs, qxt, sxt, space(fq.fp8bq_quantize_int8_t_workspace_size(n, H))),
            (fq.fp8bq_gemm_int8, qdt, sdt, qxt, sxt, dw, space(fq.fp8bq_gemm_int8_workspace_size(N, H, padded))),
            (fq.fp8bq_linear_int8, self.x, qw[:N], sw[:N], lin, space(fq.fp8bq_linear_int8_workspace_size(T, N, H))),
            (fq.fp8bq_orthogonalize, self.w.view(E, N, H), [(3.4445, -4.7750, 2.0315)] * 2, 1e-7, o,
             space(fq.fp8bq_orthogonalize_workspace_size(E, N, H))),
        ]

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.logits, self.x, self.w):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    def direct(self):
        """What the calls give, as copies."""
        for fn, *args in self.calls:
            fn(*args)
        torch.cuda.synchronize()
        return [t.clone() for t in self.outputs]

    def soil(self):
        for t in self.outputs:
            t.fill_(3)


def same(chain, want):
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(chain.outputs, want))


def test_prepared_calls():
    say("prepared routing, 8 bits, ortho")
    chain = Chain()
    assert {fn.__name__ for fn, *_ in chain.calls} == {n for n in dir(fq) if n.startswith("fp8bq_") and not n.endswith("_size") and any(
        s in n for s in ("int8", "route", "expert_rows", "gather_rows", "combine_rows", "orthogonalize"))}
    launches = [fq.prepare(*c) for c in chain.calls]
    for seed in (1, 2, 3):
        chain.fill(seed)
        want = chain.direct()
        for _ in range(2):
            chain.soil()
            for launch in launches:
                launch()
            assert same(chain, want)


def test_two_streams_at_once():
    """Two chains of different sizes, their launches interleaved on two streams: what each gives alone."""
    say("routing, 8 bits, ortho on two streams")
    chains = [Chain(), Chain(T=300, k=3, E=8, H=256, N=192, seed=5)]
    want = [c.direct() for c in chains]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for c in chains:
            c.soil()
        torch.cuda.synchronize()
        for calls in zip(*(c.calls for c in chains)):
            for s, (fn, *args) in zip(streams, calls):
                with torch.cuda.stream(s):
                    fn(*args)
        assert all(same(c, w) for c, w in zip(chains, want))


def test_captured_chain():
    """The chain in a graph, replayed on new values with eager work between the replays."""
    say("routing, 8 bits, ortho captured")
    chain = Chain(T=150, k=2)
    chain.direct()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for fn, *args in chain.calls:
            fn(*args)
    for seed in (4, 5, 6):
        chain.fill(seed)
        want = chain.direct()
        chain.soil()
        graph.replay()
        assert same(chain, want)
