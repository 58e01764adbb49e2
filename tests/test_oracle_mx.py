"""The MXFP4 oracle against the format's own facts: the sixteen values, ties, saturation, scale rule."""

import numpy as np
import pytest

from oracle import mx


def block(*vals, amax=None):
    b = np.zeros((1, 32), np.float32)
    b[0, :len(vals)] = vals
    return b


def test_every_value_of_the_format_is_kept():
    grid = np.concatenate([mx.GRID, -mx.GRID]).astype(np.float32)
    for e in (-100, -3, 0, 5, 100):
        x = np.zeros((1, 32), np.float32)
        x[0, :16] = np.ldexp(grid, e)
        code, scale = mx.quant_mx_rows(x)
        assert scale[0, 0] == e + 127
        assert np.array_equal(code[0, :16], np.arange(16))
        assert np.array_equal(mx.mx_values(code, scale), x)


@pytest.mark.parametrize("x,want", [(0.25, 0), (0.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (3.5, 4), (5.0, 4),
                                    (0.2500001, 0.5), (0.7499999, 0.5), (7.9, 6), (6.5, 6), (7.0, 6)])
def test_ties_go_to_even_codes_and_large_values_saturate(x, want):
    for sign in (1, -1):
        code, scale = mx.quant_mx_rows(block(4.0 if x < 4 else 4.0, sign * x))  # amax in [4, 8): scale 1
        assert scale[0, 0] == 127
        assert mx.mx_values(code, scale)[0, 1] == sign * want


@pytest.mark.parametrize("amax,byte", [(1.0, 125), (1.9999, 125), (2.0, 126), (4.0, 127), (2.0 ** 127, 252),
                                       (np.finfo(np.float32).max, 252), (2.0 ** -124, 1), (2.0 ** -125, 0),
                                       (2.0 ** -126, 0), (2.0 ** -149, 0), (0.0, 0), (np.inf, 255), (-np.inf, 255),
                                       (np.nan, 255)])
def test_scale_bytes(amax, byte):
    assert mx.quant_mx_rows(block(0.0, amax))[1][0, 0] == byte


def test_error_bound_and_packing():
    x = np.random.default_rng(0).standard_normal((7, 100)).astype(np.float32)
    code, scale = mx.quant_mx_rows(x)
    assert code.shape == (7, 128) and scale.shape == (7, 4)
    v = mx.mx_values(code, scale)
    # half a step: 1/4 of 2^e below 2, 1/2 below 4, 1 below 6, and up to 2 where 6 .. 8 saturates
    e = np.ldexp(1.0, scale.astype(int) - 127).repeat(32, 1)[:, :100]
    assert np.all(np.abs(v[:, :100] - x) <= np.maximum(0.25 * e, np.where(np.abs(x) > 6 * e, np.abs(x) - 6 * e,
                                                                         np.abs(x) / 4)))
    assert not v[:, 100:].any()
    assert np.array_equal(mx.unpack(mx.pack(code)), code)
    w = mx.scale_words(scale[:, :3])
    assert w.shape == (1, 7, 4) and np.array_equal(w[0, :, :3], scale[:, :3]) and not w[0, :, 3].any()
