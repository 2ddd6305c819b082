"""zr_quantize_fp8 on the GPU: codes and scales bit for bit those of a plain form,
for every type, format, grouping, alignment and edge, and nothing written
outside its matrices."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from fp8_util import E4M3, E5M2, Guarded, groups, quantize
from gpu_util import device, say

pytestmark = pytest.mark.gpu


def source(rows, cols, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if kind == "spread":  # magnitudes over the whole range of the type, zeros among them
        span = 120.0 if dtype == torch.bfloat16 else 15.0
        x = x * torch.exp2((torch.rand(rows, cols, generator=g) * 2 - 1) * span)
        x = torch.where(torch.rand(rows, cols, generator=g) < 0.2, torch.zeros(()), x)
        x = x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max)
    return x.to(dtype)


def run(x, codes, block_rows, want_q=True, want_t=True, ld=None, ldq=None, ldqt=None, offset=0):
    rows, cols = x.shape
    src = Guarded(rows, cols, x.dtype, ld, offset, fill=x)
    tall = (rows, cols) if block_rows == 1 else (groups(rows), groups(cols))
    q = Guarded(rows, cols, codes, ldq, offset) if want_q else None
    s = Guarded(tall[0], groups(cols), torch.uint8) if want_q else None
    qt = Guarded(cols, rows, codes, ldqt, offset) if want_t else None
    st = Guarded(tall[1], groups(rows), torch.uint8) if want_t else None
    view = lambda m: m.view if m is not None else None  # noqa: E731
    flat = lambda m: m.view.reshape(-1) if m is not None else None  # noqa: E731
    zr.zr_quantize_fp8(src.view, view(q), flat(s), view(qt), flat(st), block_rows=block_rows)
    torch.cuda.synchronize()
    for m in (src, q, s, qt, st):
        if m is not None:
            m.check()
    bits = lambda m: m.view.contiguous().view(torch.uint8).cpu() if m is not None else None  # noqa: E731
    return bits(q), bits(s), bits(qt), bits(st)


def check(x, codes, block_rows, got):
    q, s, qt, st = got
    if q is not None:
        wq, ws = quantize(x, codes, block_rows)
        assert torch.equal(s, ws), "scales"
        assert torch.equal(q, wq), "codes"
    if qt is not None:
        wq, ws = quantize(x.t().contiguous(), codes, block_rows)
        assert torch.equal(st, ws), "transposed scales"
        assert torch.equal(qt, wq), "transposed codes"


SIZES = [(1, 1), (1, 128), (1, 4096), (3, 127), (5, 129), (16, 512), (127, 100), (128, 128), (129, 257), (200, 384),
         (300, 1000), (1, 70_001), (1111, 8)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols, dtype):
    device()
    for codes in (E4M3, E5M2):
        for block_rows in (1, 128):
            for kind in ("normal", "spread"):
                x = source(rows, cols, dtype, rows * 1000 + cols, kind)
                check(x, codes, block_rows, run(x, codes, block_rows))
                check(x, codes, block_rows, run(x, codes, block_rows, want_t=False))
    x = source(rows, cols, dtype, 5)
    check(x, E4M3, 1, run(x, E4M3, 1, want_q=False))
    check(x, E4M3, 128, run(x, E4M3, 128, want_q=False))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("ld,ldq,ldqt,offset", [(264, 256, 144, 0), (264, 264, 136, 8), (257, 256, 130, 0),
                                                (256, 251, 144, 0), (264, 256, 137, 0), (250, 250, 130, 1)])
def test_strides_and_alignment(block_rows, ld, ldq, ldqt, offset):
    device()
    x = source(130, 250, torch.bfloat16, 7)
    for want_t in (False, True):
        check(x, E4M3, block_rows, run(x, E4M3, block_rows, True, want_t, ld, ldq, ldqt, offset))


@pytest.mark.parametrize("codes", [E4M3, E5M2])
def test_every_bf16_value(codes):
    """Every finite bf16 pattern as a group's largest value (beside fractions of it) and
    under a larger one, so that every rounding, subnormal code and scale occurs."""
    device()
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    top = torch.cat([bits, bits + 0x8000]).to(torch.int16).view(torch.bfloat16)
    f = torch.linspace(-1.0, 1.0, 128).double()
    x = (top.double()[:, None] * f).float().to(torch.bfloat16)
    x[:, 64] = top
    check(x, codes, 1, run(x, codes, 1, want_t=False))
    # the same values in one group with a fixed largest magnitude
    for big in (448.0, 57344.0, 1.0, 2.0 ** -100):
        some = top[top.abs() <= big]
        x = torch.zeros(-(-some.numel() // 127), 128, dtype=torch.bfloat16)
        x[:, 1:] = torch.nn.functional.pad(some, (0, x.shape[0] * 127 - some.numel())).view(-1, 127)
        x[:, 0] = big
        check(x, codes, 1, run(x, codes, 1, want_t=False))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_zeros_infinities_and_nan(block_rows, dtype):
    """A group of zeros has the smallest scale; a group with an infinity or a NaN is NaN
    as a whole, and no other group is touched by it."""
    device()
    x = source(300, 400, dtype, 11)
    x[5] = 0
    x[140:270, 130:260] = 0
    x[7, 3], x[290, 399], x[131, 129], x[250, 5] = float("inf"), float("nan"), float("-inf"), -float("nan")
    got = run(x, E4M3, block_rows)
    check(x, E4M3, block_rows, got)
    assert int((got[1] == 255).sum()) == (4 if block_rows == 1 else len({(0, 0), (2, 3), (1, 1), (1, 0)}))


def test_empty():
    dev = device()
    for shape in ((0, 128), (5, 0)):
        q = torch.empty(shape, dtype=E4M3, device=dev)
        zr.zr_quantize_fp8(torch.empty(shape, dtype=torch.bfloat16, device=dev), q,
                           torch.empty(0, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()


def test_flat_shard_scales_are_row_scales():
    """A flat shard quantized as one row gives the codes and scales of its rows, where the
    rows are whole groups."""
    device()
    x = source(96, 1024, torch.bfloat16, 13)
    flat, rows = run(x.reshape(1, -1), E4M3, 1, want_t=False), run(x, E4M3, 1, want_t=False)
    assert torch.equal(flat[0].reshape(-1), rows[0].reshape(-1))
    assert torch.equal(flat[1].reshape(-1), rows[1].reshape(-1))


def test_past_two_billion_elements():
    """Elements and codes past 2^31 of one long row and of a strided matrix."""
    dev = device()
    n = (1 << 31) + 128 * 5 + 8
    src = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    tail = source(1, 4096 + 8, torch.bfloat16, 17)[0]
    src[-tail.numel():] = tail.to(dev)
    q = torch.empty(n, dtype=E4M3, device=dev)
    s = torch.empty(groups(n), dtype=torch.uint8, device=dev)
    say("one row of", n)
    zr.zr_quantize_fp8(src, q, s)
    k = 128 * 30 + 8  # whole groups and the short last one
    wq, ws = quantize(tail[None, -k:], E4M3)
    assert torch.equal(q[-k:].view(torch.uint8).cpu(), wq[0]) and torch.equal(s[-31:].cpu(), ws[0])
    ld = (1 << 29) + 64
    m = src.as_strided((4, 256), (ld, 1), n - 3 * ld - 256)
    out = [torch.empty(sh, dtype=t, device=dev) for sh, t in (((4, 256), E4M3), ((4, 2), torch.uint8),
                                                             ((256, 4), E4M3), ((256, 1), torch.uint8))]
    zr.zr_quantize_fp8(m, *out)
    check(m.cpu().contiguous(), E4M3, 1, [o.view(torch.uint8).cpu() for o in out])


@pytest.mark.parametrize("block_rows,want_t", [(1, False), (1, True), (128, True)])
def test_capped_grid(monkeypatch, block_rows, want_t):
    device()
    x = source(700, 1500, torch.bfloat16, 19)
    full = run(x, E4M3, block_rows, want_t=want_t)
    for cap in ("8", "24"):
        monkeypatch.setenv("ZR_MAX_GRID", cap)
        got = run(x, E4M3, block_rows, want_t=want_t)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, full)), cap
