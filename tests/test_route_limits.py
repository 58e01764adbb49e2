"""The largest number of choices that the header allows (T k < 2^31), without a GPU: sizes just inside it reach the device
check, the next token is refused."""

import pytest
import torch

from test_route_checks import DEVICE, SHAPE, P, back, combine, combine_back, gather, route

INSIDE = [(k, (2 ** 31 - 1) // k) for k in (1, 2, 3, 5, 6, 7)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: checks the no-device path")
@pytest.mark.parametrize("k,T", INSIDE)
def test_most_choices(k, T):
    far = 1 << 42
    at = [P(0, far * i) for i in range(8)]
    route_ = lambda T: route(x=at[0], bias=at[1], e=at[2], w=at[3], T=T, k=k, E=64, ldx=64)
    back_ = lambda T: back(dw=at[0], x=at[1], e=at[2], dx=at[3], T=T, k=k, E=64, ldx=64, lddx=64)
    gather_ = lambda T: gather(x=at[0], s=at[1], out=at[2], T=T, k=k, H=8, ldx=8, ldo=8)
    combine_ = lambda T: combine(y=at[0], r=at[1], w=at[2], out=at[3], T=T, k=k, H=8, ldy=8, ldo=8)
    combine_back_ = lambda T: combine_back(d=at[0], y=at[1], r=at[2], w=at[3], s=at[4], dy=at[5], dw=at[6], T=T, k=k, H=8, ldd=8,
                                           ldy=8, ldg=8)
    for call in (route_, back_, gather_, combine_, combine_back_):
        assert call(T) == DEVICE and call(T + 1) == SHAPE
