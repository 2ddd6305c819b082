"""zr_grad_norm, zr_clip_grads and the clipped AdamW steps on the GPU.

Tolerances.  A square of a 16-bit or fp32 value is exact in fp64, sums are of terms that
are not negative: each addition on the longest path adds half a step, 2^-53 relative.  At
least 1024 sums run side by side over a tile, so a path has at most n / 1024 additions, and
at most 64 more where the sums of lanes, waves and workgroups meet (and one for each batch
of the list).  Norm and factor are fp64 until they are rounded to fp32: half a step, 2^-24.
Clipped gradients and the AdamW states are held to the exact bits: the first are one fp32
product rounded once, the others what zr_adamw_step gives for grad_scale * factor.
"""
import math
import threading

import numpy as np
import pytest
import torch

import oracle
import zero_sharded_optimizer_zr_amd as zr
from gpu_util import device, u16

pytestmark = pytest.mark.gpu
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
HP = dict(lr=5e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
inf, nan = float("inf"), float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cut(sizes, dtype, seed, offset=0, gap=0, std=1e-3):
    """Tensors of the sizes, one behind another in a buffer (`gap` elements between them) that
    starts `offset` elements past an allocation; the buffer between them is 7."""
    total = offset + sum(sizes) + gap * len(sizes) + 64
    flat = torch.full((total,), 7.0, dtype=dtype, device="cuda")
    out, at, g = [], offset, gen(seed)
    for n in sizes:
        t = flat[at:at + n]
        t.copy_(torch.randn(n, generator=g, device="cuda") * std)
        out.append(t)
        at += n + gap
    return out, flat


def norm(tensors, clip=None, ws=None, **kw):
    clip = clip if clip is not None else zr.clip_record()
    zr.zr_grad_norm(tensors, clip, ws if ws is not None else zr.grad_norm_workspace(), **kw)
    return clip


def values(clip):
    return clip[0].item(), clip.view(F32)[2].item(), clip.view(F32)[3].item()


def exact_sum(tensors):
    return math.fsum(x for t in tensors if t.numel() for x in t.double().square().cpu().tolist())


def record(norm_, factor):
    r = torch.tensor([norm_ * norm_, 0.0], dtype=torch.float64, device="cuda")
    r.view(F32)[2:] = torch.tensor([norm_, factor], device="cuda")
    return r


LISTS = [[1], [7], [8], [2047], [2048], [4096] * 3, [16384], [16385], [65535], [65537], [0, 5, 0, 1], [200_001],
         [4096] * 65, [1 + (i * 7919) % 3001 for i in range(500)], [3] * 230 + [300_000] + [9] * 230, [5_000_011, 1, 33]]


@pytest.mark.parametrize("dtype", [BF, FP16, F32])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm(sizes, dtype):
    device()
    tensors, _ = cut(sizes, dtype, len(sizes) + max(sizes))
    total, n, f = values(norm(tensors, max_norm=1e-3))
    want = exact_sum(tensors)
    assert abs(total - want) <= (sum(sizes) / 1024 + 64 + len(sizes) / 64) * 2.0 ** -53 * want
    root = math.sqrt(want)
    assert abs(n - root) <= 2.0 ** -23 * root
    factor = min(1.0, 1e-3 / (root + 1e-6))
    assert abs(f - factor) <= 2.0 ** -23 * factor


@pytest.mark.parametrize("dtype", [BF, FP16, F32])
def test_same_bits_at_any_address_and_grid(dtype, monkeypatch):
    device()
    sizes = [100_003, 1, 4096, 77, 40_000, 900_001]
    want = None
    for offset, gap, cap in [(0, 0, None), (1, 0, None), (3, 1, None), (8, 5, None), (0, 0, "8"), (5, 3, "24")]:
        if cap:
            monkeypatch.setenv("ZR_MAX_GRID", cap)
        tensors, _ = cut(sizes, dtype, 5, offset, gap)
        got = norm(tensors, max_norm=0.5).view(torch.int64).tolist()
        want = want or got
        assert got == want, (offset, gap, cap)


def test_empty_lists_and_accumulation():
    device()
    a, _ = cut([5000, 12], BF, 1)
    b, _ = cut([70_000], F32, 2)
    sa, sb = values(norm(a))[0], values(norm(b))[0]
    rec = norm(a, max_norm=1e-3)
    norm(b, rec, max_norm=1e-3, accumulate=True)
    assert values(rec)[0] == sb + sa  # two fp64 values added once
    assert values(norm([])) == (0.0, 0.0, 1.0)
    # after an all-reduce: norm and factor of what the record holds
    rec[0] = 16.0
    norm([], rec, max_norm=1.0, eps=0.0, accumulate=True)
    assert values(rec) == (16.0, 4.0, 0.25)
    norm([b[0][:0]], rec, max_norm=8.0, eps=0.0, accumulate=True)
    assert values(rec) == (16.0, 4.0, 1.0)
    # a new sum does not depend on what the record held
    rec.fill_(nan)
    norm(a, rec)
    assert values(rec)[0] == sa


def test_scales():
    device()
    x = torch.full((100,), 3.0, dtype=FP16, device="cuda")
    ls = zr.loss_scale_record()
    zr.zr_loss_scale_init(ls, 8.0)
    assert values(norm([x], max_norm=1.0, eps=0.0, ls=ls))[1:] == (3.75, float(np.float32(1 / 3.75)))
    assert values(norm([x], max_norm=1.0, eps=0.25, grad_scale=-0.5))[1:] == (15.0, float(np.float32(1 / 15.25)))
    assert values(norm([x], max_norm=1.0, grad_scale=0.0))[1:] == (0.0, 1.0)
    assert ls.tolist()[2] == 0


@pytest.mark.parametrize("dtype", [BF, FP16, F32])
def test_extremes(dtype):
    """Neither the largest nor the smallest values leave the sum; infinities and NaN show."""
    device()
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    sub = low * torch.finfo(dtype).eps  # the smallest subnormal
    for v in (top, low, sub):
        x = torch.full((3000,), v, dtype=dtype, device="cuda")
        total, n, f = values(norm([x], max_norm=1.0, eps=0.0))
        assert abs(total - 3000 * v * v) <= 1e-12 * 3000 * v * v
        root = math.sqrt(3000) * v
        assert n == (inf if root > torch.finfo(F32).max else pytest.approx(root, rel=2.0 ** -23, abs=2.0 ** -150))
        assert f == pytest.approx(min(1.0, 1 / root), rel=2.0 ** -23, abs=2.0 ** -150)
    for bad in (inf, -inf, nan):
        for at in (0, 2999, 1700):
            x = torch.ones(3000, dtype=dtype, device="cuda")
            x[at] = bad
            ls = zr.loss_scale_record()
            zr.zr_loss_scale_init(ls, 2.0)
            total, n, f = values(norm([x], max_norm=1.0, ls=ls))
            assert ls.tolist()[2] == 1
            if math.isnan(bad):
                assert math.isnan(total) and math.isnan(n) and math.isnan(f)
            else:
                assert (total, n, f) == (inf, inf, 0.0)
    assert values(norm([x]))[2] == 1.0  # no bound: never clipped


def test_below_the_bound_nothing_is_clipped():
    device()
    x = torch.full((16,), 0.25, dtype=BF, device="cuda")  # norm 1
    assert values(norm([x], max_norm=1.0, eps=0.0))[1:] == (1.0, 1.0)
    assert values(norm([x], max_norm=1.5))[1:] == (1.0, 1.0)
    assert values(norm([torch.zeros(9, device="cuda")], max_norm=1.0, eps=0.0)) == (0.0, 0.0, 1.0)


def test_past_32_bits():
    """2^31 + 77 elements in one tensor: every part of it counts."""
    device()
    n = 2 ** 31 + 77
    x = torch.zeros(n, dtype=BF, device="cuda")
    places = [0, 1, 2 ** 30 + 3, 2 ** 31 - 1, 2 ** 31, n - 1]
    for i, p in enumerate(places):
        x[p] = 2.0 ** i
    assert values(norm([x]))[0] == sum(4.0 ** i for i in range(6))
    zr.zr_clip_grads([x], record(2.0, 0.5))
    assert [x[p].item() for p in places] == [2.0 ** (i - 1) for i in range(6)]


# ------------------------------------------------------------------- clipping ----

@pytest.mark.parametrize("dtype", [BF, FP16, F32])
@pytest.mark.parametrize("offset,gap", [(0, 0), (1, 0), (5, 3), (64, 1), (63, 7)])
def test_clip_bits(dtype, offset, gap, monkeypatch):
    device()
    for cap, sizes in ((None, [1, 100_003, 16384, 0, 77]), ("8", [300_001, 5]), (None, [1 + (i * 31) % 97 for i in range(700)])):
        if cap:
            monkeypatch.setenv("ZR_MAX_GRID", cap)
        tensors, flat = cut(sizes, dtype, offset + gap, offset, gap, std=1.0)
        before = flat.clone()
        factor = 0.3712345
        want, at = before.clone(), offset
        for n in sizes:
            want[at:at + n] = (before[at:at + n].float() * np.float32(factor).item()).to(dtype)
            at += n + gap
        zr.zr_clip_grads(tensors, record(1.0, factor))
        assert torch.equal(flat, want)
        if cap:
            monkeypatch.delenv("ZR_MAX_GRID")


@pytest.mark.parametrize("dtype", [BF, FP16, F32])
def test_clip_special_factors(dtype):
    device()
    g = gen(3)
    kind = {2: torch.int16, 4: torch.int32}[torch.empty(0, dtype=dtype).element_size()]
    x = torch.randint(-2 ** 15, 2 ** 15 - 1, (5000,), generator=g, device="cuda").to(kind).view(dtype)
    before = x.view(kind).clone()
    zr.zr_clip_grads([x], record(0.5, 1.0))
    assert torch.equal(x.view(kind), before)  # every pattern, NaN payloads among them
    x = torch.randn(5000, generator=g, device="cuda").to(dtype)
    x[17], x[18] = inf, nan
    y = x.clone()
    zr.zr_clip_grads([x], record(inf, 0.0))
    assert torch.equal(x.isnan(), ~y.isfinite()) and bool((x[y.isfinite()] == 0).all())
    zr.zr_clip_grads([y], record(nan, nan))
    assert bool(y.isnan().all())


# ---------------------------------------------------------------------- AdamW ----

def state(n, dtype, seed, offsets=(0, 0, 0, 0, 0), scale=1.0):
    g = gen(seed)
    place = lambda x, o: torch.cat([torch.full((o,), 5.0, dtype=x.dtype, device="cuda"), x,  # noqa: E731
                                    torch.full((64,), 5.0, dtype=x.dtype, device="cuda")])
    r = lambda std: torch.randn(n, generator=g, device="cuda") * std  # noqa: E731
    raw = [place((r(1e-3) * scale).to(dtype), offsets[0]), place(r(0.02), offsets[1]), place(r(1e-4), offsets[2]),
           place(torch.rand(n, generator=g, device="cuda") * 1e-6, offsets[3]), place(torch.zeros(n, dtype=dtype, device="cuda"), offsets[4])]
    return [x[o:o + n] for x, o in zip(raw, offsets)], raw


def bits(x):
    return x.view(torch.int16 if x.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("dtype", [BF, FP16])
@pytest.mark.parametrize("n", [1, 3, 4, 67, 1000, 4099, 300_001])
@pytest.mark.parametrize("offsets", [(0, 0, 0, 0, 0), (4, 4, 4, 4, 4), (13, 13, 13, 13, 13), (1, 0, 2, 3, 5)])
def test_adamw_is_the_step_with_the_factor_in_its_scale(dtype, n, offsets):
    device()
    for param, grad_scale, factor in ((True, 1.0, 0.37), (True, 0.25, 0.918273), (False, 1.0, 1.0)):
        a, raw_a = state(n, dtype, n, offsets, 1024.0 if dtype == FP16 else 1.0)
        b, raw_b = state(n, dtype, n, offsets, 1024.0 if dtype == FP16 else 1.0)
        rec = record(2.0, factor)
        f32 = rec.view(F32)[3].item()
        ls = zr.loss_scale_record()
        zr.zr_loss_scale_init(ls, 1024.0)
        args_a, args_b = [*a[:4], a[4] if param else None], [*b[:4], b[4] if param else None]
        if dtype == FP16:
            zr.zr_adamw_step_f16(*args_a, ls, step=7, grad_scale=grad_scale * f32, **HP)
            zr.zr_adamw_step_clip_f16(*args_b, ls, rec, step=7, grad_scale=grad_scale, **HP)
        else:
            zr.zr_adamw_step(*args_a, step=7, grad_scale=grad_scale * f32, **HP)
            zr.zr_adamw_step_clip(*args_b, rec, step=7, grad_scale=grad_scale, **HP)
        for x, y in zip(raw_a, raw_b):
            assert torch.equal(bits(x), bits(y))


def test_adamw_against_the_oracle():
    device()
    n = 50_021
    (g, th, m, v, p), _ = state(n, BF, 9)
    host = [u16(g), *(t.cpu().numpy().copy() for t in (th, m, v)), np.zeros(n, np.uint16)]
    rec = norm([g], max_norm=0.1)
    f = values(rec)[2]
    assert 0.4 < f < 0.5
    zr.zr_adamw_step_clip(g, th, m, v, p, rec, step=3, grad_scale=0.5, **HP)
    oracle.adamw(*host, step=3, grad_scale=0.5 * f, **HP)
    for got, want in zip((th, m, v), host[1:4]):
        assert np.array_equal(got.cpu().numpy().view(np.uint32), want.view(np.uint32))
    assert np.array_equal(u16(p), host[4])


def test_adamw_f16_skips_on_overflow():
    """The norm sees the infinity; the step leaves everything as it is, as zr_adamw_step_f16 does."""
    device()
    (g, th, m, v, p), raw = state(10_001, FP16, 4, scale=1024.0)
    g[5000] = inf
    ls = zr.loss_scale_record()
    zr.zr_loss_scale_init(ls, 1024.0)
    rec = norm([g], max_norm=1.0, ls=ls)
    before = [x.clone() for x in raw]
    zr.zr_adamw_step_clip_f16(g, th, m, v, p, ls, rec, step=1, **HP)
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(raw, before))
    zr.zr_loss_scale_update(ls)
    assert ls.view(F32)[0].item() == 512.0 and ls.tolist()[1:] == [0, 0, 1]


def test_adamw_grid_cap(monkeypatch):
    device()
    for dtype in (BF, FP16):
        for offsets in ((0, 0, 0, 0, 0), (1, 0, 2, 3, 5)):
            a, _ = state(70_001, dtype, 6, offsets)
            b, _ = state(70_001, dtype, 6, offsets)
            ls = zr.loss_scale_record()
            zr.zr_loss_scale_init(ls, 1.0)
            call = (lambda s: zr.zr_adamw_step_clip_f16(*s, ls, record(2.0, 0.4), step=2, **HP)) if dtype == FP16 else \
                (lambda s: zr.zr_adamw_step_clip(*s, record(2.0, 0.4), step=2, **HP))  # noqa: B023
            call(a)
            monkeypatch.setenv("ZR_MAX_GRID", "8")
            call(b)
            monkeypatch.delenv("ZR_MAX_GRID")
            assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


# ------------------------------------------------------------------- together ----

def test_ranks_agree_with_the_whole_model():
    """Two ranks' shares of one model: sums of the slices added as an all-reduce would, the
    persistent tensors counted once; norm and factor are the whole gradient's, and the clipped
    steps are the unsharded ones."""
    device()
    numels = [300_001, 512, 150_000, 1024]
    lay = zr.zr_layout_create(numels, 2)
    info = zr.zr_layout_query(lay)
    grads, _ = cut(numels, BF, 12)
    whole = values(norm(grads, max_norm=0.25))
    slices, recs = [], []
    for r in range(2):
        b, e = zr.zr_layout_rank_range(lay, r)
        s = torch.empty(e - b, dtype=BF, device="cuda")
        zr.zr_pack(lay, [g if g.numel() >= 100_000 else None for g in grads], s, b, e)
        slices.append(s)
        recs.append(norm([s]))
    total = recs[0][0] + recs[1][0]
    small = zr.tensor_list([g for g in grads if g.numel() < 100_000])
    for rec in recs:
        rec[0] = total
        norm(small, rec, max_norm=0.25, accumulate=True)
    assert torch.equal(recs[0].view(torch.int64), recs[1].view(torch.int64))
    assert values(recs[0])[0] == pytest.approx(whole[0], rel=1e-12)
    assert values(recs[0])[1:] == pytest.approx(whole[1:], rel=2.0 ** -22)
    factor = values(recs[0])[2]
    assert factor < 1
    # one rank's clipped step against clipping in memory first
    s, rec = slices[0], recs[0]
    assert info["shard"] == s.numel()
    st = [torch.zeros(s.numel(), device="cuda") for _ in range(3)]
    st2 = [x.clone() for x in st]
    zr.zr_adamw_step_clip(s, *st, None, rec, step=1, **HP)
    zr.zr_clip_grads([s], rec)
    zr.zr_adamw_step(s, *st2, None, step=1, **HP)
    # the clipped gradient's rounding to bf16, half a step, is all that differs in m
    assert bool(((st[1] - st2[1]).abs() <= 2.0 ** -8 * 1.01 * st[1].abs() + 1e-30).all())


class Clipped:
    """reduce -> norm -> clipped AdamW of one shard, with buffers of its own."""

    def __init__(self, n, seed):
        g = gen(seed)
        self.contribs = [(torch.randn(n, generator=g, device="cuda") * 1e-3).to(BF) for _ in range(4)]
        self.grad = torch.empty(n, dtype=BF, device="cuda")
        self.st = [torch.randn(n, generator=g, device="cuda") * 0.02, torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
        self.param = torch.empty(n, dtype=BF, device="cuda")
        self.rec, self.ws = zr.clip_record(), zr.grad_norm_workspace()
        self.list = zr.tensor_list([self.grad[:n // 3], self.grad[n // 3:]])

    def run(self, step, stream=None):
        zr.zr_reduce_slice(self.contribs, self.grad, stream=stream)
        zr.zr_grad_norm(self.list, self.rec, self.ws, max_norm=0.05, stream=stream)
        zr.zr_adamw_step_clip(self.grad, *self.st, self.param, self.rec, step=step, stream=stream, **HP)
        zr.zr_clip_grads(self.list, self.rec, stream=stream)

    def outputs(self):
        return [x.clone() for x in (*self.st, self.param, self.grad, self.rec.view(torch.int64))]


@pytest.mark.parametrize("n", [3001, 700_001])
def test_captured_step_replays(n):
    device()
    eager, rec, other = Clipped(n, 1), Clipped(n, 1), Clipped(n, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        zr.zr_graph_capture_begin()
        rec.run(1)
        graph = zr.zr_graph_capture_end()
        zr.zr_graph_capture_begin()
        other.run(1)
        second = zr.zr_graph_capture_end()
    assert zr.zr_graph_info(graph)[1] == 1
    noise = torch.ones(1 << 20, device="cuda")
    for t in range(1, 6):
        for x, y in zip(eager.contribs, rec.contribs):
            x.mul_(1.25)
            y.copy_(x)
        eager.run(t)
        torch.cuda.synchronize()
        zr.zr_graph_set_adamw(graph, step=t, **HP)
        zr.zr_graph_launch(graph, side)
        zr.zr_graph_launch(second, side)
        side.synchronize()
        for x, y in zip(eager.outputs(), rec.outputs()):
            assert torch.equal(x, y), t
        noise.add_(1).sum().item()


def test_streams_and_threads_at_once():
    device()
    want = []
    for i in range(3):
        c = Clipped(200_000 + i, 20 + i)
        c.run(1)
        c.run(2)
        want.append(c.outputs())
    runs = [Clipped(200_000 + i, 20 + i) for i in range(3)]
    torch.cuda.synchronize()
    errors = []

    def work(c):
        try:
            s = torch.cuda.Stream()
            c.run(1, s)
            c.run(2, s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, w in zip(runs, want):
        assert all(torch.equal(x, y) for x, y in zip(c.outputs(), w))
