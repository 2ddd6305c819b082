"""zr_matmul_fp8 on the GPU with scales that start at any byte, as those of a tensor in a
gathered buffer do: the kernels read them in words or 16 bytes at a time.  Bytes around
the scales stand for NaN, so that one read from there shows."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from fp8_util import E4M3, E5M2, groups
from gpu_util import device, say
from test_gpu_matmul_fp8 import check, operand, run

pytestmark = pytest.mark.gpu

# split waves, two teams, the 128 x 128 ring (one and several tiles a workgroup), 256 x 256 (16-bit outputs);
# groups of the summed axis: 1, 3, 4, 5, 8, 9, 16, 17
SIZES = [(5, 200, 700), (70, 300, 1000), (300, 4100, 100), (300, 4100, 300), (250, 4100, 512), (390, 4100, 600),
         (250, 4100, 1040), (300, 4100, 2048), (200, 4100, 2100), (1500, 2050, 100), (1500, 2050, 300), (1500, 2050, 400),
         (1500, 2050, 1000), (1500, 2050, 1152), (2900, 2950, 300), (2900, 2950, 400), (2900, 2950, 600), (2900, 2950, 1024),
         (2900, 2950, 1152), (5000, 5300, 300)]


def moved(s, offset):
    """The scales in the middle of bytes of 255, `offset` bytes past a multiple of 256."""
    raw = torch.full((256 + offset + s.numel() + 256,), 255, dtype=torch.uint8, device="cuda")
    assert raw.data_ptr() % 256 == 0
    view = raw[256 + offset:256 + offset + s.numel()].view(s.shape)
    view.copy_(s)
    return view


@pytest.mark.parametrize("m,n,k", SIZES)
def test_scales_at_any_byte(m, n, k):
    device()
    lk = groups(k) * 128
    for block_rows, codes, dtype in ((1, E4M3, torch.bfloat16), (128, E5M2, torch.bfloat16), (128, E4M3, torch.float32),
                                     (1, E5M2, torch.float32)):
        a, sa = operand(m, k, codes, 1, m + k, lk, size=0.2)
        b, sb = operand(n, k, E4M3, block_rows, n + k, lk, size=0.2)
        want = run(a, sa, b, sb, block_rows, dtype).clone()
        check(want, a, sa, b, sb, block_rows)
        for at_a, at_b in ((0, 1), (1, 0), (1, 2), (2, 3), (3, 1), (3, 3), (7, 13)):
            say(m, n, k, block_rows, codes, dtype, at_a, at_b)
            assert torch.equal(run(a, moved(sa, at_a), b, moved(sb, at_b), block_rows, dtype), want)


def test_pieces_of_a_gathered_buffer():
    """Tensors of a flat buffer quantized as one row, at offsets whose scales start at every byte
    of a word, as the operand of products that each LDS kernel takes."""
    dev = device()
    shapes = [(1100, 384), (600, 640), (2100, 128), (4100, 640), (2050, 640), (2950, 640)]
    numels = [r * c for r, c in shapes]
    g = torch.Generator(device="cuda").manual_seed(2)
    # 128 elements before the first tensor and between two: each starts a byte further
    starts, at = [], 128
    for x in numels:
        starts.append(at)
        at += x + 128
    flat = (torch.randn(at, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    codes, scales = torch.empty(at, dtype=E4M3, device=dev), torch.empty(at // 128, dtype=torch.uint8, device=dev)
    zr.zr_quantize_fp8(flat, codes, scales)
    seen = set()
    for start, numel, (n, k) in zip(starts, numels, shapes):
        q = codes[start:start + numel].view(n, k)
        s = scales[start // 128:(start + numel) // 128].view(n, groups(k))
        alone_q, alone_s = q.clone(), s.clone()
        seen.add(s.data_ptr() % 4)
        for tokens in (300, 1500, 2900):
            x, sx = operand(tokens, k, E4M3, 1, tokens)
            outs = []
            for qq, ss in ((q, s), (alone_q, alone_s)):
                outs.append(torch.empty(tokens, n, dtype=torch.bfloat16, device=dev))
                zr.zr_matmul_fp8(x.view, sx, qq, ss, outs[-1])
            assert torch.equal(*outs) and not bool(outs[0].isnan().any())
    assert seen == {0, 1, 2, 3}
