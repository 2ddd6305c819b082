"""Plain forms of the 8-bit floating-point operators for the tests, in 64 bits
or on exact bits, on the CPU or the GPU, and guarded matrices."""
import torch

GROUP = 128
E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
TOP = {E4M3: 8, E5M2: 15}          # largest value: 1.75 * 2^TOP
# largest rounding error relative to the value: half a step
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32, E4M3, E5M2)}
# largest rounding error near zero: half of the smallest subnormal
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def groups(n):
    return -(-n // GROUP)


def blocks_amax(x, block_rows):
    """Largest magnitude of each group of 128 along a row (or 128 x 128 block) of x (64 bits)."""
    rows, cols = x.shape
    tall = -(-rows // block_rows) * block_rows
    p = torch.nn.functional.pad(x.abs(), (0, groups(cols) * GROUP - cols, 0, tall - rows))
    return p.view(tall // block_rows, block_rows, groups(cols), GROUP).amax(dim=(1, 3))


def scale_bytes(amax, codes):
    """E8M0 bytes: the smallest e >= -127 with amax <= 1.75 * 2^TOP * 2^e; 255 for non-finite."""
    amax = amax.double()
    part, e = torch.frexp(amax)
    e = e - 1 - TOP[codes] + (part > 0.875).to(e.dtype)
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(min=-127))
    return torch.where(torch.isfinite(amax), e + 127, torch.full_like(e, 255)).to(torch.uint8)


def spread(s, shape, block_rows):
    """Scale values (64 bits) of every element of a matrix of `shape`."""
    v = torch.exp2(s.view(torch.uint8).double() - 127)
    v = torch.where(s.view(torch.uint8) == 255, torch.full_like(v, float("nan")), v)
    v = v.repeat_interleave(block_rows, 0)[:shape[0]]
    return v.repeat_interleave(GROUP, 1)[:, :shape[1]]


def quantize(x, codes, block_rows=1):
    """(codes as bytes, scale bytes) of a bf16 or fp16 matrix.  x * 2^-e is exact in
    fp32 (a 16-bit x, and what underflows there is far below half a code), so torch's
    conversion rounds it once."""
    s = scale_bytes(blocks_amax(x.double(), block_rows), codes)
    v = (x.double() / spread(s, x.shape, block_rows)).float()
    q = v.to(codes).view(torch.uint8)
    return torch.where(torch.isnan(v), torch.full_like(q, 0x7f), q), s


def values(q, s, block_rows=1):
    """Values (64 bits) that codes and scales stand for."""
    return q.double() * spread(s, q.shape, block_rows)


class Guarded:
    """A matrix inside a larger allocation of a pattern nobody writes: row distance
    `ld`, first element at `offset`, 256 bytes behind; `check()` asserts that
    everything outside the matrix still holds the pattern."""

    def __init__(self, rows, cols, dtype, ld=None, offset=0, fill=None, device="cuda"):
        self.ld = ld or max(1, cols)
        size = torch.empty(0, dtype=dtype).element_size()
        self.size, self.rows, self.cols, self.offset = size, rows, cols, offset
        total = (offset + max(0, rows - 1) * self.ld + cols) * size + 256
        self.raw = torch.full((-(-total // 4) * 4,), 0xA5, dtype=torch.uint8, device=device)
        n = self.raw.numel() // size * size
        self.view = self.raw[:n].view(dtype).as_strided((rows, cols), (self.ld, 1), offset)
        if fill is not None:
            self.view.view(torch.uint8).copy_(fill.to(device).contiguous().view(torch.uint8)) if size == 1 \
                else self.view.copy_(fill)

    def check(self):
        keep = torch.ones_like(self.raw, dtype=torch.bool)
        keep.as_strided((self.rows, self.cols * self.size), (self.ld * self.size, 1), self.offset * self.size).fill_(False)
        assert bool((self.raw[keep] == 0xA5).all()), "write outside the matrix"
