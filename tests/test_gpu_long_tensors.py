"""Tensors past 2^32 bytes and calls of more rows than one launch has threads for: routing, the experts' rows and the
8-bit operators give there what they give for a part of the rows alone."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
MANY = (1 << 26) + 5


def ends(n, at=1 << 24):
    """Some rows around multiples of 2^24 and at both ends."""
    near = [r for c in range(0, n + 1, at) for r in range(c - 3, c + 3)] + list(range(n - 5, n))
    return torch.tensor(sorted({r for r in near if 0 <= r < n}), device="cuda")


def test_routing_of_many_tokens():
    say("route", MANY)
    x = torch.empty(MANY, 8, dtype=BF16, device="cuda").normal_()
    rows = ends(MANY)
    experts, w = fq.route_experts(x, 2, "softmax")
    some = fq.route_experts(x[rows].contiguous(), 2, "softmax")
    assert torch.equal(experts[rows], some[0]) and torch.equal(w[rows], some[1])
    dx = fq.route_experts_backward(w, x, experts, "softmax")
    assert torch.equal(dx[rows], fq.route_experts_backward(w[rows].contiguous(), x[rows].contiguous(), some[0], "softmax"))


def test_codes_of_many_rows():
    say("quantize_int8", MANY)
    x = torch.empty(MANY, 16, dtype=BF16, device="cuda").normal_()
    rows = ends(MANY)
    q, s = fq.quantize_int8(x)
    qs, ss = fq.quantize_int8(x[rows].contiguous())
    assert torch.equal(q[rows], qs) and torch.equal(s[rows], ss)


def test_rows_past_4_gib():
    T, k, E, H = 70000, 4, 16, 8192
    say("rows", T, k, H)
    x = torch.empty(T, H, dtype=BF16, device="cuda").normal_()
    g = torch.Generator().manual_seed(1)
    experts = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    offsets, rows, slots = fq.expert_rows(experts, E)
    xs = fq.gather_rows(x, slots, k)
    some = ends(T * k, 1 << 17)
    assert torch.equal(xs[some], x[(slots[some] // k).long()])
    out = fq.combine_rows(xs, rows, w)
    tokens = ends(T, 1 << 15)
    want = (w[tokens].double().sum(1, keepdim=True) * x[tokens].double())
    # k products and sums in FP32 of values of one sign: (k + 1) 2^-24, and the rounding to BF16
    assert bool(((out[tokens].double() - want).abs() <= want.abs() * (2.0 ** -8 + 6 * 2.0 ** -24)).all())
    dy, dw = fq.combine_rows_backward(x, xs, rows, w, slots)
    choice = slots[some].long()
    want = w.flatten()[choice].unsqueeze(1) * x[choice // k].float()
    assert torch.equal(dy[some], want.to(BF16))
    dot = (x[tokens].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    # a sum of H / 256 terms a thread, of 64 lanes and of four waves, all positive
    assert bool(((dw[tokens].double() - dot).abs() <= dot * (H // 256 + 16) * 2.0 ** -24).all())


def test_products_past_4_gib():
    say("gemm_int8 rows past 4 GiB")
    g = torch.Generator().manual_seed(2)
    M, N, K = 300000, 72, 16384  # the codes
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    b = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sa, sb = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    rows = ends(M, 1 << 17)
    got = fq.gemm_int8(a, sa, b, sb, out_dtype=F32)[rows]
    assert torch.equal(got, fq.gemm_int8(a[rows].contiguous(), sa[rows].contiguous(), b, sb, out_dtype=F32))
    del a
    M, N, K = 70000, 16408, 64  # the output
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    b = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sa, sb = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    rows = ends(M, 1 << 15)
    got = fq.gemm_int8(a, sa, b, sb, out_dtype=F32)[rows]
    assert torch.equal(got, fq.gemm_int8(a[rows].contiguous(), sa[rows].contiguous(), b, sb, out_dtype=F32))


@pytest.mark.parametrize("R,C", [(33, 1 << 20), ((1 << 20), 40)])
def test_orthogonalize_the_longest_sides(R, C):
    """Rows of one direction each that stay what they are: G with orthogonal rows (columns) of equal length, whose singular
    values are all 1 / sqrt(m) of the norm and go through the polynomial alike."""
    say("ortho", R, C)
    m = min(R, C)
    g = torch.zeros(R, C, device="cuda")
    i = torch.arange(m, device="cuda")
    far = (max(R, C) - 1) // m
    if R < C:
        g[i, i * far] = 3.0
    else:
        g[i * far, i] = 3.0
    got = fq.orthogonalize(g)
    # First-order bound of the error e of s: A = s^2 and P = b A + c A^2 are rounded to 11 bits (u = 2^-11 at most), and P
    # meets the first half of X (u again); what is there already goes through the step's slope.  2% for the second order
    # and the FP32 sums; the result's rounding to BF16 is 2^-8.
    s, e, u = m ** -0.5, 0.0, 2.0 ** -11
    a, b, c = 3.4445, -4.7750, 2.0315
    for _ in range(5):
        A = s * s
        P = b * A + c * A * A
        e = 1.02 * (abs(a + 3 * b * A + 5 * c * A * A) * e + s * u * (2 * abs(P) + abs(b + 2 * c * A) * A))
        s = a * s + P * s
    want = torch.where(g != 0, s, 0.0).to(torch.float64)
    assert bool(((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + e / s)).all())
