"""The accuracy that the orthogonalization's header states, against Newton-Schulz steps in float64.

A result y is the exact w plus an error e, rounded to BF16, so |y - w| <= |e| + half the step of BF16 at w (where w and w + e
lie on two sides of a power of two, y is that power at most that far).  What |y - w| has beyond that half step is held to
2^-14 of the norm of w.  Where that comes from: every operand is held in 22 bits and sums in FP32; the same scheme on the CPU
is off by 5 10^-7 with exact sums and by up to 2.3 10^-6 (five steps) and 5 10^-6 (ten) with FP32 ones on the matrices
below, and a factor of twelve is left for the order of the sums."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
MUON = (3.4445, -4.7750, 2.0315)


def exact(g, coefficients, eps=1e-7):
    out = []
    for x in g.to(F64):
        turned = x.shape[0] > x.shape[1]
        x = x.t() if turned else x
        x = x / (x.square().sum().sqrt() + eps)
        for a, b, c in coefficients:
            A = x @ x.t()
            x = a * x + (b * A + c * (A @ A)) @ x
        out.append(x.t() if turned else x)
    return torch.stack(out)


def hold(got, g, coefficients=(MUON,) * 5, eps=1e-7, bound=2.0 ** -14):
    torch.cuda.synchronize()
    for y, w in zip(got.to(F64), exact(g, coefficients, eps)):
        half_step = torch.ldexp(torch.ones_like(w), torch.frexp(w).exponent - 9)  # w = f 2^e, 1/2 <= f < 1: steps of 2^(e - 8)
        beyond = ((y - w).abs() - half_step).clamp(min=0.0)
        off = float(beyond.norm()) / float(w.norm())
        print("off by", off, flush=True)
        assert off <= bound


def normal(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def orthogonal_rows(m, n):
    """Equal singular values."""
    return torch.linalg.qr(normal(n, m, seed=m).to(F64))[0].t().to(F32).unsqueeze(0)


def low_rank(m, n, r):
    u = normal(1, m, r, seed=2) / torch.arange(1, r + 1, device="cuda").sqrt()
    v = normal(1, n, r, seed=3)
    return (u.unsqueeze(2) * v.unsqueeze(1)).sum(3) + 0.2 * normal(1, m, n, seed=4)


MATRICES = {
    "random": [normal, (1, 256, 2048), (1, 64, 1024), (1, 32, 1024), (3, 32, 32), (2, 64, 64), (4, 64, 256), (5, 8, 8), (7, 2, 3),
               (1, 512, 384), (1, 1000, 700), (1, 300, 5000), (2, 1408, 1100)],
    "equal": [orthogonal_rows, (400, 1024), (4, 1024), (130, 130), (1, 33)],
    "low": [low_rank, (512, 384, 32), (700, 2050, 7), (96, 96, 1)],
}
CASES = [(kind, shape) for kind, (_, *shapes) in MATRICES.items() for shape in shapes]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,shape", CASES, ids=[f"{k}-{'x'.join(map(str, s))}" for k, s in CASES])
def test_five_steps(kind, shape, dtype):
    say("ortho accuracy", kind, shape, dtype)
    g = MATRICES[kind][0](*shape).to(dtype)
    hold(fq.orthogonalize(g), g)
    turned = g.transpose(1, 2).contiguous()
    hold(fq.orthogonalize(turned), turned)


@pytest.mark.parametrize("shape", [(512, 384), (40, 100)])
def test_identity(shape):
    say("ortho accuracy identity", shape)
    g = torch.eye(*shape, device="cuda").unsqueeze(0)
    hold(fq.orthogonalize(g), g)


@pytest.mark.parametrize("steps", [1, 2, 10])
def test_other_numbers_of_steps(steps):
    say("ortho accuracy steps", steps)
    for dtype in (F32, BF16):
        g = normal(1, 256, 1024, seed=5).to(dtype)
        hold(fq.orthogonalize(g, steps=steps), g, (MUON,) * steps)


STRONG = [((10.0, 0.0, 0.0), (0.1, 0.0, 0.0)),                     # the singular value goes to 10 and back to 1
          ((15.0, 0.0, 0.0), (0.05, 0.0, 0.0), (1.5, -0.5, 0.0)),
          ((14.0, 0.0, 0.0), (0.25, 0.9, 0.001)),                  # a polynomial of 215 at 14
          ((0.5, -16.25, 0.0), (0.06, 0.0, 0.0))]                  # and one below zero, the value at -15.75


@pytest.mark.parametrize("coefficients", STRONG)
@pytest.mark.parametrize("shape", [(1, 1), (1, 40), (40, 1), (50, 70), (300, 128)])
def test_up_to_the_stated_limits(shape, coefficients):
    """Singular values up to 15 and polynomials up to 215, where one row has all of the norm, so that a single entry of A is
    the largest singular value's square and one of X may be that value."""
    say("ortho limits", shape, coefficients)
    g = torch.zeros(1, *shape, device="cuda")
    g[0, shape[0] // 2] = normal(shape[1], seed=7)
    hold(fq.orthogonalize(g, steps=len(coefficients), coefficients=list(coefficients)), g, coefficients)
    g = torch.zeros(1, *shape, device="cuda")
    g[0, shape[0] // 2, shape[1] // 3] = 3.0
    hold(fq.orthogonalize(g, steps=len(coefficients), coefficients=list(coefficients)), g, coefficients)


@pytest.mark.parametrize("steps", [1, 5, 12])
@pytest.mark.parametrize("size", [1e-9, 1e-12, 1e-17, 1e-18, 1e-20, 1e-30])
def test_norms_far_below_eps(size, steps):
    """X = G / (|G| + eps) is then tiny, and the steps take it up again by about 3.44 each, to one after enough of them."""
    say("ortho small", size, steps)
    for dtype in (F32, BF16):
        g = (normal(4, 128, 256, seed=9) * size).to(dtype)
        g[1] *= 1e-6
        g[2] = 0.0
        g[3] = normal(128, 256, seed=10)
        y = fq.orthogonalize(g, steps=steps)
        assert not y[2].any() and bool((y[[0, 1, 3]] != 0).any(2).all())
        near_all = g[[0, 1, 3]]
        hold(y[[0, 1, 3]], near_all, (MUON,) * steps)
        wide = (normal(1, 1000, 700, seed=11) * size).to(dtype)
        hold(fq.orthogonalize(wide, steps=steps), wide, (MUON,) * steps)


@pytest.mark.parametrize("eps", [1e-3, 1.0, 1e4, 1e30])
def test_large_eps(eps):
    say("ortho eps", eps)
    each = [(3.0, -3.2, 1.2), (0.01, 0.0, 0.0), (20.0, -5.0, 7.0), (3.4445, -4.7750, 2.0315)]
    g = normal(1, 90, 333, seed=12)
    hold(fq.orthogonalize(g, steps=4, coefficients=each, eps=eps), g, each, eps)


def test_steps_that_leave_nothing():
    say("ortho nothing")
    g = normal(2, 70, 80, seed=13)
    for first in ((0.0, 0.0, 0.0), (1e-300, 0.0, 0.0)):
        y = fq.orthogonalize(g, steps=3, coefficients=[first, MUON, MUON])
        assert not y.any()
