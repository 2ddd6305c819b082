"""Results of zr_matmul_fp8's 256 x 256 tiles on the GPU after long sums: whole and cut vectors,
odd row distances and addresses, accumulation."""
import pytest
import torch

from fp8_util import E4M3, E5M2
from gpu_util import device, say
from test_gpu_matmul_fp8 import check, operand, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1920, 2048, 2064, 2432])
@pytest.mark.parametrize("m,n", [(2817, 2945), (2900, 2951), (5000, 5300)])
def test_stores(m, n, k):
    device()
    for codes, dtype, pad, offset in ((E4M3, torch.bfloat16, 0, 0), (E5M2, torch.bfloat16, 3, 1), (E4M3, torch.float16, 8, 5)):
        lk = -(-k // 128) * 128
        a, sa = operand(m, k, codes, 1, m + k, lk, size=0.2)
        b, sb = operand(n, k, E4M3, 128, n + k, lk, size=0.2)
        say(m, n, k, codes, dtype)
        check(run(a, sa, b, sb, 128, dtype, n + pad, offset), a, sa, b, sb, 128)
        start = torch.randn(m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
        check(run(a, sa, b, sb, 128, dtype, n + pad, offset, start), a, sa, b, sb, 128, start)
