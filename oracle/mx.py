"""Microscaled 4-bit operands (OCP MXFP4): blocks of 32, E2M1 codes, E8M0 scales.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Per block: e = max(floor(log2(amax)) - 2, -127); each code is the value of the E2M1 grid nearest to x 2^-e, at
equal distance the one with an even code, values past 6 going to 6, the sign kept.  Found by comparing exact
distances in float64 over the eight magnitudes.  A block with a NaN or an infinity has the scale byte 255.
"""

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quant_mx_rows(x):
    """x float32 [R, C], blocks of 32 along C (the last filled up with zeros).  Returns codes uint8 [R, Cp]
    (one per value, Cp = C rounded up to 32) and scale bytes uint8 [R, Cp / 32]."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    Cp = -(-C // 32) * 32
    v = np.zeros((R, Cp))
    v[:, :C] = x
    v = v.reshape(R, Cp // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1))
    mant, ex = np.frexp(amax)
    e = np.maximum(np.where(amax > 0, ex - 1 - 2, -127), -127)
    y = np.abs(np.ldexp(np.where(np.isfinite(v), v, 0.0), -e[..., None]))
    dist = np.abs(y[..., None] - GRID)
    near = dist.min(-1, keepdims=True)
    order = np.where(np.arange(8) % 2 == 0, 0, 1)  # even codes first among the nearest
    code = np.argmin(np.where(dist == near, order, 9), -1).astype(np.uint8)
    code |= (np.signbit(v).astype(np.uint8) << 3)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(R, Cp), scale


def mx_values(code, scale):
    """float64 values of codes [R, Cp] with scale bytes [R, Cp / 32]."""
    code = np.asarray(code)
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(int) - 127))
    return (v.reshape(code.shape[0], -1, 32) * s[..., None]).reshape(code.shape)


def pack(code):
    """Two codes a byte, the even element in the low half."""
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(q):
    c = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = q & 15, q >> 4
    return c


def scale_words(scale):
    """[R, nb] bytes as [ceil(nb / 4), R, 4], zeros past nb."""
    R, nb = scale.shape
    w = np.zeros((R, -(-nb // 4) * 4), np.uint8)
    w[:, :nb] = scale
    return np.ascontiguousarray(w.reshape(R, -1, 4).transpose(1, 0, 2))
