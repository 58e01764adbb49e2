"""Sizes at which the planner takes each of the 8-bit products' tiles, with the tile it is to take (256 compute units): held to
the planner on the host, so that none of them can fall back to other tiles unseen, and run on the GPU against float64 (the
roundings as in test_gpu_int8.py)."""

import os
import shutil
import subprocess

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (M, N, K, tile rows, tile columns, parts of the contraction, three stages): rows, columns and contractions that end
# inside a tile and a stage
DENSE = [(300, 400, 528, 64, 64, 1, 1), (300, 400, 4112, 64, 64, 6, 1), (1025, 2900, 144, 64, 64, 1, 0),
         (1100, 1100, 16400, 128, 128, 5, 0), (2049, 2500, 144, 128, 128, 1, 0), (4099, 2570, 272, 256, 192, 1, 0),
         (4081, 2701, 16, 256, 192, 1, 0), (8100, 8100, 144, 256, 256, 1, 0)]
# (tokens of each expert, N, K, tile rows, tile columns)
GROUPED = [([40] * 8, 1408, 528, 64, 64), ([513, 385, 0, 255, 384] * 7, 1408, 528, 128, 128),
           ([1500, 0, 257, 129, 1280, 256], 2570, 528, 256, 192), ([700] * 12 + [1, 0, 129, 255], 953, 144, 256, 192),
           ([1030] * 8, 2570, 144, 256, 256)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    csrc = os.path.join(ROOT, "fp8_blockwise_quantized_amd", "csrc")
    exe = str(tmp_path_factory.mktemp("plan") / "planned_int8")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-I", csrc, os.path.join(ROOT, "tests", "csrc", "planned_int8.cpp"),
                        os.path.join(csrc, "plan.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = {k: v for k, v in os.environ.items() if k != "FP8BQ_GEMM_TILE"}

    def ask(*args):
        r = subprocess.run([exe], input=" ".join(str(a) for a in args) + "\n", capture_output=True, text=True, env=env)
        assert r.returncode == 0, r.stderr
        return tuple(int(v) for v in r.stdout.split())

    return ask


@pytest.mark.parametrize("M,N,K,rows,cols,parts,deep", DENSE)
def test_planned(plan, M, N, K, rows, cols, parts, deep):
    for linear in (0, 1):
        assert plan(linear, 0, M, N, K) == (rows, cols, parts, deep)


@pytest.mark.parametrize("counts,N,K,rows,cols", GROUPED)
def test_planned_grouped(plan, counts, N, K, rows, cols):
    for linear in (0, 1):
        assert plan(linear, len(counts), sum(counts), N, K)[:2] == (rows, cols)


def operands(M, rows_b, K):
    g = torch.Generator().manual_seed(M + rows_b + K)
    a, b = (torch.randint(-128, 128, (n, K), generator=g, dtype=torch.int8).cuda() for n in (M, rows_b))
    sa, sb = (torch.rand(n, generator=g).cuda() * 0.05 + 1e-4 for n in (M, rows_b))
    return a, sa, b, sb


def exact(a, sa, b, sb):
    return (a.double() @ b.double().t()) * sa.double().unsqueeze(1) * sb.double()


def close(got, want, before=None):
    """The sum made FP32 and two scales: three roundings of 2^-24 at most; one of 2^-8 to BF16, one of 2^-24 when added."""
    limit = want.abs() * 3.01 * 2.0 ** -24
    if before is not None:
        want = want + before.double()
        limit = limit + want.abs() * 1.01 * 2.0 ** -24
    if got.dtype == torch.bfloat16:
        limit = limit + want.abs() * 2.0 ** -8
    assert bool(((got.double() - want).abs() <= limit).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [c[:3] for c in DENSE])
def test_products(M, N, K):
    say("int8 tiles", M, N, K)
    a, sa, b, sb = operands(M, N, K)
    want = exact(a, sa, b, sb)
    for out in (torch.bfloat16, torch.float32):
        close(fq.gemm_int8(a, sa, b, sb, out_dtype=out), want)
    c = torch.randn(M, N, device="cuda")
    close(fq.gemm_int8(a, sa, b, sb, out=c.clone(), accumulate=True), want, c)
    wide = torch.full((M + 1, N + 3), 7.0, device="cuda")  # rows that start off 16 bytes, and what lies around them
    fq.gemm_int8(a, sa, b, sb, out=wide[:M, :N])
    close(wide[:M, :N], want)
    assert bool((wide[M:] == 7.0).all()) and bool((wide[:, N:] == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [c[:3] for c in GROUPED], ids=lambda v: f"{len(v)}of{sum(v)}" if isinstance(v, list) else None)
def test_grouped_products(counts, N, K):
    say("int8 grouped tiles", counts[:6], N, K)
    E, T = len(counts), sum(counts) + 5
    off = torch.tensor([2] + counts).cumsum(0).cuda()
    a, sa, b, sb = operands(T, E * N, K)
    o = off.tolist()
    y = [torch.full((T, N), 5.0, dtype=out, device="cuda") for out in (torch.bfloat16, torch.float32)]
    for t in y:
        fq.grouped_gemm_int8(a, sa, off, b, sb, out=t)
    for e in range(E):
        r, w = slice(o[e], o[e + 1]), slice(e * N, (e + 1) * N)
        want = exact(a[r], sa[r], b[w], sb[w])
        for t in y:
            close(t[r], want)
    for t in y:
        assert bool((t[:o[0]] == 5.0).all()) and bool((t[o[-1]:] == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 70, 12288), (1, 70, 12304), (3, 70, 4096), (1, 70, 65392), (16, 70, 3952)])
def test_rows_quantized_in_the_product(M, N, K):
    """The longest rows that a workgroup quantizes for itself, and longer ones."""
    say("int8 skinny", M, N, K)
    _, _, w, sw = operands(M, 2 * N, K)
    x = torch.randn(M, K, device="cuda")
    q, s = fq.quantize_int8(x)
    assert torch.equal(fq.linear_int8(x, w, sw), fq.gemm_int8(q, s, w, sw))
    off = torch.tensor([0, M // 2, M], device="cuda")
    assert torch.equal(fq.grouped_linear_int8(x, off, w, sw), fq.grouped_gemm_int8(q, s, off, w, sw))
