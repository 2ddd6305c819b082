"""How zr_matmul_fp8 adds, on the GPU: fp32 outputs add every product in fp32; 16-bit outputs
add each run of 8 products to 13 bits below the largest, and no less."""
import pytest
import torch

from fp8_util import E4M3, E5M2, Guarded, groups, values
from gpu_util import device, say
from test_gpu_matmul_fp8 import check, operand, run

pytestmark = pytest.mark.gpu

# every shape of a split wave's tile, two teams, the 128 x 128 ring, 256 x 256 (16-bit outputs)
SIZES = [(3, 200, 1000), (16, 300, 640), (16, 11008, 256), (60, 3900, 400), (100, 4096, 384), (1100, 1030, 391), (250, 4100, 1000),
         (1500, 2050, 400), (2900, 2950, 400)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_every_code_and_scale_with_16_bit_outputs(m, n, k):
    """Random bytes as codes (no NaN) and scales over a wide range: subnormal codes, zeros and the
    largest ones go through the scaled instructions."""
    device()
    for codes, bad in ((E4M3, 0x7f), (E5M2, 0x7c)):
        for block_rows in (1, 128):
            g = torch.Generator(device="cuda").manual_seed(6)
            bytes_ = lambda r, c, hi=256: torch.randint(0, hi, (r, c), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
            qa, qb = bytes_(m, k), bytes_(n, k)
            qa[(qa & 0x7f) >= bad] = 0x38
            qb[(qb & 0x7f) == 0x7f] = 0
            tall = n if block_rows == 1 else groups(n)
            sa, sb = 100 + bytes_(m, groups(k), 40), 110 + bytes_(tall, groups(k), 30)
            a, b = Guarded(m, k, codes, groups(k) * 128, 0, qa), Guarded(n, k, E4M3, groups(k) * 128, 0, qb)
            say(m, n, k, codes, block_rows)
            check(run(a, sa, b, sb, block_rows, torch.bfloat16), a, sa, b, sb, block_rows)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_fp32_outputs_add_in_fp32(m, n, k):
    """In every run of 8 one product of 2^s and one of 2^(s - 16), the rest zeros: their sums are
    exact in fp32 (at most 125 runs: 24 bits) and lose the smaller ones where runs are aligned to
    13 bits.  2^-8 is a subnormal e4m3 code."""
    device()
    for codes in (E4M3, E5M2):
        one = {E4M3: 0x38, E5M2: 0x3c}[codes]
        small = {E4M3: 0x02, E5M2: 0x1c}[codes]  # 2^-8
        g = torch.Generator().manual_seed(m)
        runs = -(-k // 8)
        qa = torch.zeros(m, runs, 8, dtype=torch.uint8)
        even, odd = (2 * torch.randint(0, 4, (m, runs, 1), generator=g) + i for i in (0, 1))
        qa.scatter_(2, even, one)
        qa.scatter_(2, odd, small)
        qa = qa.view(m, -1)[:, :k].contiguous()
        qb = torch.tensor([0x38, 0x02], dtype=torch.uint8).repeat(n, -(-k // 2))[:, :k].contiguous()
        a, b = Guarded(m, k, codes, groups(k) * 128, 0, qa.cuda()), Guarded(n, k, E4M3, groups(k) * 128, 0, qb.cuda())
        sa = torch.full((m, groups(k)), 127, dtype=torch.uint8, device="cuda") + (torch.arange(m, device="cuda") % 5).to(torch.uint8)[:, None]
        sb = torch.full((n, groups(k)), 120, dtype=torch.uint8, device="cuda") + (torch.arange(n, device="cuda") % 7).to(torch.uint8)[:, None]
        want = values(a.view, sa) @ values(b.view, sb).t()
        assert torch.equal(want.float().double(), want)
        assert torch.equal(run(a, sa, b, sb, 1, torch.float32), want.float())


@pytest.mark.parametrize("m,n,k", [(64, 64, 4096), (64, 128, 1024), (40, 100, 11008)])
def test_16_bit_outputs_lose_no_more_than_stated(m, n, k):
    """Each row times itself minus its own permutation: the exact sum is 0, so that what comes
    out is what adding has lost, whatever the rounding of the result.  A product of two codes
    loses its part below 2^-12 of the power of two at or below its run's largest (13 bits, and one
    because the largest product is below twice that power): itself if it is smaller than that.
    The losses' sum, and k half steps of fp32, bound each element.  On normal data the stated
    1.4e-5 of a product, for the two halves and with a factor of 2 for the spread of the data:
    2 sqrt(2) 1.4e-5."""
    device()
    perm = torch.randperm(k, generator=torch.Generator().manual_seed(1)).cuda()
    for codes in (E4M3, E5M2):
        a, sa = operand(m, k, codes, 1, 5)
        b, sb = operand(n, k, E4M3, 1, 6)
        # one scale a row, so that codes may change places
        sa[:] = sa.amax(1, keepdim=True)
        sb[:] = sb.amax(1, keepdim=True)
        qa, qb = a.view.view(torch.uint8), b.view.view(torch.uint8)
        a2 = Guarded(m, 2 * k, codes, None, 0, torch.cat([qa, qa[:, perm] ^ 0x80], 1))
        b2 = Guarded(n, 2 * k, E4M3, None, 0, torch.cat([qb, qb[:, perm]], 1))
        sa2, sb2 = sa.repeat(1, 2).contiguous(), sb.repeat(1, 2).contiguous()
        va, vb = values(a2.view, sa2), values(b2.view, sb2)
        bound = torch.empty(m, n, dtype=torch.float64, device="cuda")
        for i in range(m):
            p = (va[i] * vb).abs().view(n, -1, 8)
            cut = torch.exp2(torch.floor(torch.log2(p.amax(2, keepdim=True).clamp(min=2.0 ** -300))) - 12)
            bound[i] = torch.where(p < cut, p, torch.where(p % cut == 0, torch.zeros_like(p), cut)).sum((1, 2))
        bound += 2 * k * 2.0 ** -24 * (va.abs() @ vb.abs().t())
        half = va[:, :k] @ vb[:, :k].t()
        for dtype in (torch.bfloat16, torch.float16):
            got = run(a2, sa2, b2, sb2, 1, dtype).double()
            assert bool((got.abs() <= bound).all())
            lost = float(got.norm() / half.norm())
            say(m, n, k, codes, dtype, "lost", lost, "largest of its bound", float((got.abs() / bound).max()))
            assert lost <= 2 * 2 ** 0.5 * 1.4e-5
        # fp32 outputs: k steps of fp32, no more
        got = run(a2, sa2, b2, sb2, 1, torch.float32).double()
        assert bool((got.abs() <= 2 * k * 2.0 ** -23 * (va.abs() @ vb.abs().t())).all())
        say("fp32", float(got.norm() / half.norm()))
        assert float(got.norm() / half.norm()) <= 2.0 ** -21
