"""The products on the planner's larger tiles (tile_cases.py; test_planned_tiles.py holds the sizes to those tiles): every
output type, edges that end inside a tile, guards around outputs and workspaces.  Compared on the device with the
float64 product of the same codes: within 1e-4 ||a|| ||b|| (the FP32 rule of parity.py), and a BF16 output half a unit
in its last place more, 2^-8 |y|."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say
from test_gpu_grouped_split import expected, operands
from tile_cases import WGRAD

pytestmark = pytest.mark.gpu


def guarded(rows, cols, dtype):
    """A buffer of sevens and the matrix inside it."""
    big = torch.full((rows + 8, cols + 16), 7.0, dtype=dtype, device="cuda")
    return big, big[4:rows + 4, :cols]


def close(got, y, lim):
    if got.dtype == torch.bfloat16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
    return bool(torch.all((got.double() - y).abs() <= lim))


def untouched(big, inner):
    inner.fill_(7.0)
    return bool(torch.all(big == 7.0))


@pytest.mark.parametrize("name", sorted(WGRAD))
def test_grouped_weight_gradients(name):
    say("tiles wgrad", name)
    counts, N, K, _, split = WGRAD[name]
    E = len(counts)
    off, (qdyt, sdyt), (qxt, sxt) = operands(counts, N, K, 500)
    y, lim = expected(counts, qdyt, sdyt, qxt, sxt)
    size = fq.fp8bq_grouped_gemm_wgrad_workspace_size(E, qdyt.shape[1], N, K)
    assert (size > 0) == split
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(dw, space, **kw):
        fq.fp8bq_grouped_gemm_wgrad(qdyt, sdyt, fq.E5M2, qxt, sxt, fq.E4M3, off, dw, ws=space, **kw)

    for space in (ws[:size], None) if split else (None,):
        big, one = guarded(E * N, K, torch.float32)
        run(one, space)
        assert close(one, y, lim)
        start = torch.randn(E * N, K, device="cuda")
        wide, acc = guarded(E * N, K, torch.float32)
        acc.copy_(start)
        run(acc, space, accumulate=True)
        assert torch.equal(acc, start + one)  # one FP32 addition an element
        half, dw = guarded(E * N, K, torch.bfloat16)
        run(dw, space)
        assert close(dw, y, lim)
        assert untouched(big, one) and untouched(wide, acc) and untouched(half, dw)
    assert torch.all(ws[size:] == 0xFF)
