"""zr_matmul_fp8 on the GPU with elements (code * scale) past the range of bf16 and fp32: products
and sums that fp32 holds are right, whatever the elements are.  Tolerances are those
of test_gpu_matmul_fp8, whose `check` they go through."""
import pytest
import torch

from fp8_util import E4M3, E5M2, Guarded, groups, quantize
from gpu_util import device, say
from test_gpu_matmul_fp8 import check, operand, run

pytestmark = pytest.mark.gpu

# every shape of a split wave's tile, two teams, the 128 x 128 ring and (16-bit outputs) 256 x 256
SIZES = [(1, 40, 300), (16, 300, 640), (7, 4096, 512), (16, 11008, 256), (60, 3900, 400), (100, 4096, 384), (1100, 1030, 391),
         (250, 4100, 1040), (300, 400, 128), (1500, 2050, 400), (2900, 2950, 400)]


def small(rows, k, codes, block_rows, seed):
    """An operand whose elements are around 2^-24 in size."""
    return operand(rows, k, codes, block_rows, seed, groups(k) * 128, size=2.0 ** -24)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_the_quantizers_largest_codes(m, n, k):
    """The largest bf16 value rounds to the code of 2^128 (256 * 2^120, 32768 * 2^113)."""
    device()
    top = torch.finfo(torch.bfloat16).max
    for codes in (E4M3, E5M2):
        x = torch.randn(m, k, generator=torch.Generator().manual_seed(k)).to(torch.bfloat16)
        x[::2, ::3], x[1::2, 0] = top, -top
        q, s = quantize(x, codes)
        a = Guarded(m, k, codes, groups(k) * 128, 0, q)
        s = s.cuda()
        assert int(s.max()) == (247 if codes == E4M3 else 240)
        for block_rows in (1, 128):
            b, sb = small(n, k, E4M3, block_rows, n)
            for dtype in (torch.float32, torch.bfloat16):
                say(m, n, k, codes, block_rows, dtype)
                got = run(a, s, b, sb, block_rows, dtype)
                assert bool(got.isfinite().all())
                check(got, a, s, b, sb, block_rows)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_large_scales(m, n, k):
    """Scale bytes up to 254 in some groups of some rows of one operand and moderate elements in the
    other; what the rows without them give keeps its bits."""
    device()
    for codes in (E4M3, E5M2):
        a, sa = small(m, k, codes, 1, m)
        b, sb = small(n, k, E4M3, 1, n)
        plain = {t: run(a, sa, b, sb, 1, t).clone() for t in (torch.float32, torch.bfloat16)}
        g = torch.Generator().manual_seed(1)
        for which, s in (("a", sa), ("b", sb)):
            hit = (torch.rand(s.shape, generator=g) < 0.3).cuda() & (torch.arange(s.shape[0], device="cuda") % 3 == 0)[:, None]
            hit[0, 0] = True
            # e5m2 codes reach 2^7 further than e4m3 ones; the others are around 2^-24, below 2^-18
            top = 240 if which == "a" and codes == E5M2 else 247
            big = torch.where(hit, torch.randint(top, 255 - (248 - top), s.shape, generator=g).cuda().to(torch.uint8), s)
            ba, bb = (big, sb) if which == "a" else (sa, big)
            for t, before in plain.items():
                say(m, n, k, codes, which, t)
                got = run(a, ba, b, bb, 1, t)
                assert bool(got.isfinite().all())
                check(got, a, ba, b, bb, 1)
                same = ~hit.any(1)
                assert torch.equal(got[same], before[same]) if which == "a" else torch.equal(got[:, same], before[:, same])


@pytest.mark.parametrize("m,n,k", [(60, 3900, 400), (250, 4100, 1040), (1500, 2050, 400)])
def test_large_scales_of_both(m, n, k):
    """Sums past fp32's range are infinite (or, of either sign, NaN) and stay in their elements."""
    device()
    a, sa = small(m, k, E4M3, 1, m)
    b, sb = small(n, k, E4M3, 1, n)
    plain = run(a, sa, b, sb, 1, torch.float32).clone()
    sa[5, 1], sb[9, 1] = 254, 250
    got = run(a, sa, b, sb, 1, torch.float32)
    assert not bool(got[5, 9].isfinite())
    rows, cols = torch.arange(m) != 5, torch.arange(n) != 9
    assert torch.equal(got[rows][:, cols], plain[rows][:, cols])
    part_a = Guarded(1, k, E4M3, None, 0, a.view.view(torch.uint8)[5:6])
    part_b = Guarded(n - 1, k, E4M3, None, 0, b.view.view(torch.uint8)[cols])
    check(got[5:6][:, cols], part_a, sa[5:6], part_b, sb[cols], 1)


@pytest.mark.parametrize("m,n,k", [(1, 40, 600), (60, 3900, 512), (100, 4096, 512), (1100, 1030, 591), (250, 4100, 1040), (1500, 2050, 600)])
def test_groups_that_add_nothing(m, n, k):
    """Zeros of one operand under large scales of the other leave every sum as it is, from the
    smallest ones to large ones."""
    device()
    for codes in (E4M3, E5M2):
        for which in "ab":
            a, sa = operand(m, k, codes, 1, m, groups(k) * 128)
            b, sb = operand(n, k, E4M3, 1, n, groups(k) * 128)
            s, other = (sa, b) if which == "a" else (sb, a)
            rows = torch.arange(s.shape[0], device="cuda")
            s.copy_((27 + rows * 29 % 190)[:, None].expand(s.shape))  # sums from 2^-100 to 2^90
            other.view.view(torch.uint8)[:, 128:256] = 0
            want = run(a, sa, b, sb, 1, torch.float32).clone()
            s[::2, 1] = 254
            s[1::4, 1] = 240 if which == "a" and codes == E5M2 else 247
            assert torch.equal(run(a, sa, b, sb, 1, torch.float32), want)
