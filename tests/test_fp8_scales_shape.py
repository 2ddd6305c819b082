"""The binding looks at the shape of a matrix of scales: rows of another length, or of another
grouping of b, would be read at wrong places (CPU only: refused before any launch)."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
M, N, K = 6, 300, 700  # 6 groups along k, 3 blocks along n


def codes(rows, cols):
    return torch.zeros(rows, cols, dtype=E4M3)


def scales(*shape):
    return torch.zeros(*shape, dtype=E8M0)


def product(a_scales, b_scales, block_rows, n=N):
    zr.zr_matmul_fp8(codes(M, K), a_scales, codes(n, K), b_scales, torch.zeros(M, n, dtype=torch.bfloat16), b_block_rows=block_rows)


@pytest.mark.parametrize("a_scales,b_scales,block_rows,n", [
    ((M, 6), (N, 6), 128, N),        # a scale per row where one per block is asked for
    ((M, 6), (100, 6), 128, 100),    # the same with a single block
    ((M, 6), (N, 7), 1, N), ((M, 6), (3, 7), 128, N), ((M, 6), (N + 1, 6), 1, N), ((M, 6), (6, N), 1, N),
    ((M, 7), (N, 6), 1, N), ((M + 1, 7), (3, 6), 128, N)])
def test_products_refuse_scales_of_another_shape(a_scales, b_scales, block_rows, n):
    with pytest.raises(ValueError, match="_scales is"):
        product(scales(*a_scales), scales(*b_scales), block_rows, n)


@pytest.mark.parametrize("a_scales,b_scales,block_rows", [
    ((M, 6), (N, 6), 1), ((M, 6), (3, 6), 128), ((M * 6,), (N * 6,), 1), ((M * 6 + 9,), (3 * 6 + 9,), 128),
    ((1, M * 6), (1, N * 6), 1), ((M + 5, 6), (N, 6), 1)])
def test_products_take_matching_and_flat_scales(a_scales, b_scales, block_rows):
    with pytest.raises(ValueError, match="cuda"):  # past the arguments' checks
        product(scales(*a_scales), scales(*b_scales), block_rows)


def test_quantizer_and_norm():
    x = torch.zeros(5, K, dtype=torch.bfloat16)
    for make in (lambda s: zr.zr_quantize_fp8(x, codes(5, K), s), lambda s: zr.zr_quantize_fp8(x.t().contiguous(), qt=codes(5, K), scales_t=s),
                 lambda s: zr.zr_rmsnorm_fp8(x, x[0], q=codes(5, K), scales=s)):
        with pytest.raises(ValueError, match="is 5 x 8, 5 x 6 needed"):
            make(scales(5, 8))
        for good in (scales(5, 6), scales(9, 6), scales(30), scales(1, 40)):
            with pytest.raises(ValueError, match="cuda"):
                make(good)
    # a flat shard's scales may have the shape of its rows' scales
    with pytest.raises(ValueError, match="cuda"):
        zr.zr_quantize_fp8(torch.zeros(4 * 256, dtype=torch.bfloat16), torch.zeros(4 * 256, dtype=E4M3), scales(4, 2))
