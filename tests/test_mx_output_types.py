"""Output types of the MXFP4 entry points, without a GPU: BF16 and FP32 everywhere, added to the output only by the dense
product of codes (the one whose header offers it and whose binding has it); the others refuse that type as the FP8
fprop does."""

import pytest

from test_mx_checks import DEVICE, DTYPE, HAVE_GPU, gemm, linear


def test_only_the_dense_product_of_codes_is_added_to_its_output():
    assert gemm(ct=2, grouped=True) == DTYPE
    for grouped in (False, True):
        assert linear(ct=2, grouped=grouped) == DTYPE and linear(ct=2, grouped=grouped, xt=1) == DTYPE
        assert linear(ct=2, grouped=grouped, M=0) == DTYPE


@pytest.mark.skipif(HAVE_GPU, reason="fake pointers: checks the no-device path")
def test_the_others_pass():
    assert gemm(ct=2) == DEVICE
    for ct in (0, 1):
        for grouped in (False, True):
            assert gemm(ct=ct, grouped=grouped) == DEVICE and linear(ct=ct, grouped=grouped) == DEVICE
