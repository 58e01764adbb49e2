"""The planner's choices for the sizes of tile_cases.py (host only, built with g++)."""

import os
import shutil
import subprocess

import pytest

from tile_cases import MX_GROUPED, MX_SPLIT, ROWS, WGRAD, padded

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    csrc = os.path.join(ROOT, "fp8_blockwise_quantized_amd", "csrc")
    exe = str(tmp_path_factory.mktemp("plan") / "planned_tiles")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-I", csrc, os.path.join(ROOT, "tests", "csrc", "planned_tiles.cpp"),
                        os.path.join(csrc, "plan.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = {k: v for k, v in os.environ.items() if k != "FP8BQ_GEMM_TILE"}

    def ask(*args):
        r = subprocess.run([exe], input=" ".join(str(a) for a in args) + "\n", capture_output=True, text=True, env=env)
        assert r.returncode == 0, r.stderr
        return [int(v) for v in r.stdout.split()]

    return ask


@pytest.mark.parametrize("name", sorted(WGRAD))
def test_grouped_weight_gradients(plan, name):
    counts, N, K, rows, split = WGRAD[name]
    for ws in (0, 1):
        tile, _, sets = plan("grouped", 2, len(counts), padded(counts), N, K, ws)
        assert tile == rows and (sets > 0) == (split and ws == 1)


def test_which_outputs_the_caches_keep(plan):
    """BF16 outputs of 48 MB and more whose rows lie a multiple of 8 KB apart, where they fit the 256 MB cache with their
    operands (8192 x 8192 x 2048), and all below 6 MB; FP32 outputs from 100 to 320 MB and below 6; whatever is added to
    its output."""
    def past(M, N, K, out=0, ld=None):
        size = 4 if out else 2
        return plan("stores", out, size * M * N, (M + N) * K, int(size * (ld or N) % 8192 == 0)) == [1]

    assert not past(8192, 8192, 2048) and not past(8192, 4096, 2048) and not past(4096, 16384, 1024)
    assert past(8192, 8192, 2048, ld=8448) and past(8192, 7936, 2048) and not past(8192, 7936, 2048, ld=8192)
    assert past(16384, 8192, 2048) and past(4096, 4096, 4096)
    assert past(16384, 11264, 2048) and past(16384, 2048, 2048) and past(16384, 2560, 2048) and past(2048, 2048, 2048)
    assert not past(512, 2048, 2048) and not past(1, 11264, 2048)
    assert not past(8192, 8192, 2048, 1) and past(16384, 11264, 2048, 1) and past(2048, 2048, 2048, 1)
    assert not past(8192, 8192, 2048, 2) and not past(16384, 11264, 2048, 2) and not past(2048, 2048, 2048, 2)


@pytest.mark.parametrize("name", sorted(ROWS))
def test_grouped_rows(plan, name):
    counts, N, K, fprop, dgrad = ROWS[name]
    for op, rows in ((0, fprop), (1, dgrad)):
        assert plan("grouped", op, len(counts), sum(counts), N, K, 0)[0] == rows


@pytest.mark.parametrize("name", sorted(MX_GROUPED))
def test_grouped_mxfp4(plan, name):
    counts, N, K, rows = MX_GROUPED[name]
    for linear in (0, 1):
        assert plan("mx", linear, len(counts), sum(counts), N, K)[0] == rows


@pytest.mark.parametrize("M,N,K,rows,parts", MX_SPLIT)
def test_split_mxfp4(plan, M, N, K, rows, parts):
    for linear in (0, 1):
        tile, _, split = plan("mx", linear, 0, M, N, K)
        assert (tile, split) == (rows, parts)
