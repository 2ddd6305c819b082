"""Sizes past what the 8-bit operators' kernels count in are refused (CPU only)."""
import pytest

import zero_sharded_optimizer_zr_amd as zr
from test_fp8_abi import MATMUL, call

MOST = ((1 << 31) - 65) * 128  # groups of the summed axis are counted in 32 bits, a few past the last one


@pytest.mark.parametrize("k", [MOST + 1, 1 << 39, (1 << 63) - 1])
def test_products_of_too_long_rows(k):
    at = dict(a=1 << 44, b=1 << 44, a_scales=1 << 43, b_scales=1 << 42, out=1 << 41)
    assert call("zr_matmul_fp8", MATMUL, m=1, n=1, k=k, lda=k, ldb=k, ldo=1, **at) == 1
    assert "k = " in zr.zr_last_error()
