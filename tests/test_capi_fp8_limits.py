"""Sizes that a launch of the 8-bit floating-point operators cannot hold are refused before anything runs.

Pointers are never dereferenced: a call that started a kernel before its refusal would report
that kernel's failure here, where there is no GPU, instead of the size.
"""
import ctypes

import pytest

import bit_gemm_token_amd as bgt

OK = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("xtype", [0, 1, 2])
@pytest.mark.parametrize("ytype", [0, 1, 2])
@pytest.mark.parametrize("K", [1, 128, 300])
def test_linear_refused_before_its_rows(xtype, ytype, K):
    """The product's grid is past 2^32 threads, that of the rows' quantization is not."""
    assert bgt.lib().bgt_w8a8_linear_fp8(OK, xtype, K, OK, OK, 1 << 24, 1 << 18, K, OK, OK, OK, ytype, None) == bgt.BGT_ERR_SHAPE
