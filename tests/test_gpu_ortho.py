"""Orthogonalized updates against Newton-Schulz steps in float64.

What the kernels round is stated in their header: X to two halves (22 bits), of which the products take the first, A and the
polynomial to 11 bits, the result to BF16 (2^-8).  The same scheme in float64 (emulated below) says how far that takes the result; the kernels round at the same
places, at other values in the last bit, so they are held to twice the emulation's distance from the exact steps, and each
element to twelve times its root mean square (a tail of a million roundings).  An error dP of the polynomial moves element
(i, j) of X by sum_k dP[i, k] X[k, j], which grows with the size of X's column j, so the mean is also taken along each
vector of the shorter side by itself (columns of falling sizes differ a hundredfold).  In matrices of a few numbers roundings do not
average, and the last step alone may be off by 2^-11 (|b| A + 2 |c| A^2 + |P|) |x|, that is 16 times 2^-11 for A up to 1.3."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
MUON = (3.4445, -4.7750, 2.0315)


def gradient(shape, seed, kind="random"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    B, R, C = shape
    if kind == "low":  # rank 3 in noise
        u = torch.randn(B, R, 3, generator=g, device="cuda")
        v = torch.randn(B, 3, C, generator=g, device="cuda")
        x = (u.unsqueeze(3) * v.unsqueeze(1)).sum(2) + 0.02 * x
    elif kind == "decay":  # columns of falling size
        x = x / torch.arange(1, C + 1, device="cuda")
    return x


def half(t, scale):
    return (t * scale).to(torch.float16).to(F64) / scale


def steps_of(g, coefficients, eps=1e-7, emulate=False):
    out = []
    for x in g.to(F64):
        turned = x.shape[0] > x.shape[1]
        x = x.t() if turned else x
        x = x / (x.square().sum().sqrt() + eps)
        for a, b, c in coefficients:
            if emulate:
                hi = half(x, 4096.0)
                lo = half(x - hi, 4096.0)
                A = half(hi @ hi.t(), 1024.0)
                P = half(b * A + c * (A @ A), 1024.0)
                x = a * (hi + lo) + P @ hi
            else:
                A = x @ x.t()
                x = a * x + (b * A + c * (A @ A)) @ x
        out.append(x.t() if turned else x)
    return torch.stack(out)


def check(got, g, coefficients=(MUON,) * 5, eps=1e-7):
    torch.cuda.synchronize()
    want = steps_of(g, coefficients, eps)
    near = steps_of(g, coefficients, eps, emulate=True)
    assert got.dtype == BF16 and got.shape == g.shape
    for y, w, e in zip(got.to(F64), want, near):
        rms = 2.0 * float((e - w).square().mean().sqrt()) + 1e-12
        if w.numel() <= 4096:
            rms += 16 * 2.0 ** -11 * float(w.square().mean().sqrt())
        along = 2.0 * (e - w).square().mean(0 if w.shape[0] <= w.shape[1] else 1, keepdim=True).sqrt()
        off = (y - w).abs()
        beyond = (off - 2.0 ** -8 * w.abs()).clamp(min=0.0)
        assert float(beyond.square().mean().sqrt()) <= rms
        assert bool((off <= 2.0 ** -8 * w.abs() * (1 + 2.0 ** -8) + 12.0 * (rms + along)).all()), (float(off.max()), rms)


SHAPES = [(1, 1, 1), (1, 1, 9), (1, 9, 1), (1, 3, 5), (2, 64, 64), (3, 65, 130), (1, 130, 65), (2, 108, 441), (1, 441, 108),
          (8, 512, 384), (5, 128, 256), (1, 300, 9000), (1, 9000, 300), (1, 1030, 1000), (2, 777, 2050), (40, 40, 72),
          (1, 2048, 2048), (3, 1408, 2048)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["random", "low", "decay"])
def test_five_steps(shape, dtype, kind):
    say("ortho", shape, dtype, kind)
    g = gradient(shape, sum(shape), kind).to(dtype)
    check(fq.orthogonalize(g), g)


@pytest.mark.parametrize("shape", [(2, 96, 200), (1, 300, 70)])
@pytest.mark.parametrize("steps", [1, 2, 3, 7])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_other_steps_and_coefficients(shape, steps, dtype):
    say("ortho steps", shape, steps, dtype)
    g = gradient(shape, steps).to(dtype)
    check(fq.orthogonalize(g, steps=steps), g, (MUON,) * steps)
    each = [(1.5, -0.5, 0.0), (3.0, -3.2, 1.2), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0),
            (1.5, -0.5, 0.0)][:steps]
    check(fq.orthogonalize(g, steps=steps, coefficients=each), g, each)


def test_singular_vectors_stay():
    """Coefficients that converge to one: U V^T of the singular value decomposition."""
    say("ortho svd")
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.linalg.qr(torch.randn(90, 60, generator=g, device="cuda", dtype=F64))[0]
    v = torch.linalg.qr(torch.randn(60, 60, generator=g, device="cuda", dtype=F64))[0]
    x = (u * torch.linspace(0.5, 2.0, 60, device="cuda", dtype=F64)) @ v.t()
    got = fq.orthogonalize(x.to(F32), steps=12, coefficients=(1.875, -1.25, 0.375))
    # rounding to BF16, and 11-bit roundings of the last steps, which nothing amplifies: 4 of them of entries below 1/2
    assert float((got.to(F64) - u @ v.t()).abs().max()) <= 2.0 ** -9 + 4 * 2.0 ** -11


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e18, 1e37])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_magnitudes(size, dtype):
    say("ortho magnitudes", size, dtype)
    g = (gradient((2, 70, 130), 5) * 0.2).to(dtype) * size
    eps = 1e-7 if size >= 1e-12 else 1e-32
    check(fq.orthogonalize(g, eps=eps), g, eps=eps)


def test_zeros_nan_and_infinity_stay_their_own():
    say("ortho masks")
    for dtype in (BF16, F32):
        g = gradient((5, 100, 150), 6).to(dtype)
        g[1] = 0.0
        g[2, 3, 4] = float("nan")
        g[3, 99, 149] = float("inf")
        y = fq.orthogonalize(g)
        assert not y[1].any() and bool(y[2].isnan().all()) and bool(y[3].isnan().all())
        check(y[::4], g[::4])


def test_strides_guards_and_alignment():
    say("ortho strides")
    for R, C in ((100, 150), (150, 100), (67, 75)):
        for pad in (0, 1, 8, 13):
            for dtype in (BF16, F32):
                big = gradient((3, R + 2, C + pad), R + pad).to(dtype)
                g = big[:, 1:R + 1, :C]
                guard = torch.full((3, R + 2, C + pad + 1), 7.0, dtype=BF16, device="cuda")
                out = guard[:, 1:R + 1, 1:C + 1] if pad % 8 else guard[:, 1:R + 1, :C]
                fq.orthogonalize(g, out=out)
                check(out.contiguous(), g.contiguous())
                out.fill_(7.0)
                assert bool((guard == 7.0).all())
    g = gradient((1, 80, 90), 1)[0]
    assert torch.equal(fq.orthogonalize(g), fq.orthogonalize(g.unsqueeze(0))[0])
    assert torch.equal(fq.orthogonalize(g.t().contiguous()), fq.orthogonalize(g).t())


def test_deterministic_and_the_same_on_two_streams():
    say("ortho streams")
    g1, g2 = gradient((1, 1000, 3000), 1).to(BF16), gradient((4, 600, 500), 2)
    want = [fq.orthogonalize(g1), fq.orthogonalize(g2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, g in zip(streams, (g1, g2)):
            with torch.cuda.stream(s):
                got.append(fq.orthogonalize(g))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("shape", [(1, 130, 65), (1, 300, 5000), (6, 256, 128)])
def test_captured_and_replayed(shape):
    say("ortho graph", shape)
    g = gradient(shape, 1)
    fq.orthogonalize(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fq.orthogonalize(g)
    for seed in range(3):
        g.copy_(gradient(shape, 10 + seed))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, fq.orthogonalize(g))


def test_hyperball_step_along_it():
    """The chain of an optimizer step: momentum, orthogonalized, then the normalized update at a fixed radius."""
    say("ortho hyperball")
    E, R, C = 4, 128, 192
    w = gradient((E, R, C), 1).view(E * R, C).contiguous()
    m = gradient((E, R, C), 2, "low")
    o = fq.orthogonalize(m)
    radius = float(w.to(F64).norm())
    want_w, flat = w.to(F64), o.view(E * R, C)
    fq.hyperball_step(w, flat, lr=0.5, weight_decay=0.0, radius=radius)
    want_w = want_w - 0.5 * flat.to(F64) / flat.to(F64).norm()
    want_w = want_w * (radius / want_w.norm())
    torch.cuda.synchronize()
    # 2^-21 of the magnitudes that are added, as for the step alone
    limit = 2.0 ** -21 * (want_w.abs() + 0.5 * flat.to(F64).abs() / flat.to(F64).norm()) * 1.01
    assert bool(((w.to(F64) - want_w).abs() <= limit + 2.0 ** -21 * want_w.abs()).all())
    check(o, m)


def test_empty():
    say("ortho empty")
    assert fq.orthogonalize(torch.zeros(0, 3, 4, device="cuda")).shape == (0, 3, 4)
    assert fq.orthogonalize(torch.zeros(5, 0, device="cuda")).shape == (5, 0)
