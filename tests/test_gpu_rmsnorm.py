"""zr_rmsnorm_fp8 and zr_rmsnorm_backward on the GPU against the formulas in 64 bits.

Tolerances.  A sum of `cols` positive fp32 terms, kept by at least 64 lanes one
after the other and then joined in a tree, is off by at most (cols / 64 + 16) *
2^-24 relative (standard summation bound: one half step per addition on the
longest path; the squares are exact in the fused multiply-add).  rstd halves
that and adds a division, a square root and an addition: +4 half steps.  y adds
two products.  Each output then rounds once.
"""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from fp8_util import E4M3, HALF, TINY, Guarded, blocks_amax, groups, scale_bytes, spread
from gpu_util import device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def sum_bound(cols):
    return (cols / 64 + 16) * U


def data(rows, cols, dtype, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return ((r(rows, cols) * size).to(dtype), (r(rows, cols) * 2 * size).to(dtype), (1 + 0.2 * r(cols)).to(dtype),
            r(rows, cols).to(dtype), r(rows, cols).to(dtype))


def forward(x, w, residual=None, eps=1e-5, want="hyqr", ld=None, ldq=None, offset=0, in_place=None):
    rows, cols = x.shape
    t = x.dtype
    mx, mr = Guarded(rows, cols, t, ld, offset, x), Guarded(rows, cols, t, ld, offset, residual) if residual is not None else None
    mw = Guarded(1, cols, t, None, offset, w[None])
    h = Guarded(rows, cols, t, ld, offset) if "h" in want and residual is not None else None
    if in_place:
        h = mx if in_place == "x" else mr
    y = Guarded(rows, cols, t, ld, offset) if "y" in want else None
    q = Guarded(rows, cols, E4M3, ldq, offset) if "q" in want else None
    s = Guarded(rows, groups(cols), torch.uint8) if "q" in want else None
    rstd = Guarded(1, rows, torch.float32) if "r" in want else None
    view = lambda m: None if m is None else m.view  # noqa: E731
    row = lambda m: None if m is None else m.view.reshape(-1)  # noqa: E731
    zr.zr_rmsnorm_fp8(mx.view, row(mw), view(y), view(q), row(s), residual=view(mr), h=view(h), rstd=row(rstd), eps=eps)
    torch.cuda.synchronize()
    for m in (mx, mr, mw, h, y, q, s, rstd):
        if m is not None:
            m.check()
    return {"h": view(h), "y": view(y), "q": view(q), "s": view(s), "rstd": row(rstd)}


def check_forward(out, x, w, residual=None, eps=1e-5):
    rows, cols = x.shape
    t = x.dtype
    h = x if residual is None else (x.float() + residual.float()).to(t)
    if out["h"] is not None:
        assert torch.equal(out["h"], h), "h"
    hd = h.double()
    rstd = 1 / torch.sqrt(hd.pow(2).mean(1) + eps)
    b = sum_bound(cols) / 2 + 4 * U
    if out["rstd"] is not None:
        assert bool(((out["rstd"].double() - rstd).abs() <= b * rstd).all()), "rstd"
    y = hd * rstd[:, None] * w.double()
    by = b + 2 * U
    if out["y"] is not None:
        off = (out["y"].double() - y).abs()
        assert bool((off <= (HALF[t] * (1 + by) + by) * y.abs() + TINY[t]).all()), "y"
    if out["q"] is not None:
        amax = blocks_amax(y, 1)
        s = out["s"].int()
        # the scale of an amax that may be off by `by`
        low, high = (scale_bytes(amax * f, E4M3).int() for f in (1 - by, 1 + by))
        assert bool(((low <= s) & (s <= high)).all()), "scales"
        scale = spread(out["s"], y.shape, 1)
        got = out["q"].double() * scale
        bound = (HALF[E4M3] * (1 + by) + by) * y.abs() + 2.0 ** -10 * scale
        assert bool(((got - y).abs() <= bound).all()), "codes"


SIZES = [(1, 1), (1, 128), (2, 100), (3, 4096), (1, 4096), (5, 257), (64, 512), (33, 1000), (17, 1024), (9, 2048),
         (7, 3000), (6, 5000), (5, 8192), (3, 11008), (3, 16384), (2, 20000), (2, 40000), (700, 640)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward_sizes(rows, cols, dtype):
    device()
    x, res, w, _, _ = data(rows, cols, dtype, cols)
    check_forward(forward(x, w, res), x, w, res)
    check_forward(forward(x, w, None, want="q"), x, w)
    check_forward(forward(x, w, None, want="yr"), x, w)
    check_forward(forward(x, w, res, want="hq"), x, w, res)


@pytest.mark.parametrize("ld,ldq,offset", [(1008, 1000, 0), (1008, 1008, 8), (1001, 1000, 0), (1000, 1003, 0), (1000, 1000, 1)])
def test_forward_strides_and_alignment(ld, ldq, offset):
    device()
    x, res, w, _, _ = data(19, 1000, torch.bfloat16, 3)
    check_forward(forward(x, w, res, ld=ld, ldq=ldq, offset=offset), x, w, res)


@pytest.mark.parametrize("cols", [100, 1024, 4096, 20000])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_forward_in_place(into, cols):
    device()
    x, res, w, _, _ = data(21, cols, torch.bfloat16, 4)
    check_forward(forward(x, w, res, in_place=into), x, w, res)


@pytest.mark.parametrize("cols", [200, 4096, 20000])
def test_forward_zero_rows_infinities_and_nan(cols):
    """A row of zeros stays zero (eps > 0); a row with an infinity or a NaN does not reach
    another row, and every group it makes NaN says so."""
    device()
    x, res, w, _, _ = data(8, cols, torch.bfloat16, 5)
    clean = forward(x, w, want="yqr")
    bad = x.clone()
    bad[1], bad[3, 17], bad[6, cols - 1] = 0, float("nan"), float("inf")
    out = forward(bad, w, want="yqr")
    for r in (0, 2, 4, 5, 7):
        for k in ("y", "q", "s"):
            assert torch.equal(out[k][r].view(torch.uint8), clean[k][r].view(torch.uint8)), (r, k)
    assert bool((out["y"][1] == 0).all()) and bool((out["q"][1].view(torch.uint8) & 0x7f == 0).all())
    assert bool((out["s"][1] == 0).all())
    # NaN in a row: its mean is NaN, so every value is
    assert bool(out["y"][3].isnan().all()) and bool((out["s"][3] == 255).all())
    # an infinity: rstd = 0, its own product is NaN, the others are 0
    assert bool(out["y"][6, cols - 1].isnan()) and bool((out["y"][6, :cols - 1] == 0).all())
    assert out["s"][6, -1] == 255 and bool((out["s"][6, :-1] == 0).all())
    assert bool((out["q"][6].view(torch.uint8)[groups(cols) * 128 - 128:] == 0x7f).all())


def test_forward_small_and_large_magnitudes():
    device()
    for size, eps in ((1e-3, 1e-6), (1e-18, 0.0), (1e15, 1e-5)):
        x, res, w, _, _ = data(9, 1000, torch.bfloat16, 6, size)
        check_forward(forward(x, w, res, eps=eps), x, w, res, eps)


def backward(dy, h, w, rstd, dh=None, ld=None, offset=0, in_place=None, fill=None):
    rows, cols = h.shape
    t = h.dtype
    mdy, mh = Guarded(rows, cols, t, ld, offset, dy), Guarded(rows, cols, t, ld, offset, h)
    mdh = Guarded(rows, cols, t, ld, offset, dh) if dh is not None else None
    mw = Guarded(1, cols, t, None, offset, w[None])
    dx = {"dy": mdy, "dh": mdh}[in_place] if in_place else Guarded(rows, cols, t, ld, offset)
    dw = Guarded(1, cols, t, None, offset)
    ws = Guarded(1, zr.ZR_RMSNORM_PARTIALS * cols, torch.float32)
    zr.zr_rmsnorm_backward(mdy.view, mh.view, mw.view.reshape(-1), rstd, dx.view, dw.view.reshape(-1), ws.view, dh=None if mdh is None else mdh.view)
    torch.cuda.synchronize()
    for m in (mdy, mh, mdh, mw, dx, dw, ws):
        if m is not None:
            m.check()
    return dx.view, dw.view.reshape(-1)


def check_backward(got, dy, h, w, rstd, dh=None):
    dx, dw = got
    rows, cols = h.shape
    t = h.dtype
    dyd, hd, wd, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    g = dyd * wd
    # the dot's error is relative to the sum of its terms' magnitudes; +1 for each product
    dot_off = (sum_bound(cols) + 2 * U) * (g * hd).abs().mean(1, keepdim=True)
    k = r * r * (g * hd).mean(1, keepdim=True)
    want = r * (g - hd * k)
    off = r * (r * r * dot_off * hd.abs() + 6 * U * (g.abs() + (hd * k).abs()))
    if dh is not None:
        want = want + dh.double()
        off = off + 2 * U * (dh.double().abs() + want.abs())
    assert bool(((dx.double() - want).abs() <= HALF[t] * (want.abs() + off) + off + TINY[t]).all()), "dx"
    terms = dyd * hd * r
    # rows summed one after the other (at most rows / 64 + 64 in a chain), then the partial sums
    off = (rows / 64 + 64 + 512 + 4) * U * terms.abs().sum(0)
    want = terms.sum(0)
    assert bool(((dw.double() - want).abs() <= HALF[t] * (want.abs() + off) + off + TINY[t]).all()), "dweight"


def rstd_of(h, eps=1e-5):
    return torch.rsqrt(h.float().square().mean(1) + eps)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", SIZES + [(513, 256), (1025, 1000), (2000, 64), (600, 4096)])
def test_backward_sizes(rows, cols, dtype):
    device()
    _, h, w, dy, dh = data(rows, cols, dtype, cols + 1)
    rstd = rstd_of(h)
    check_backward(backward(dy, h, w, rstd), dy, h, w, rstd)
    check_backward(backward(dy, h, w, rstd, dh), dy, h, w, rstd, dh)


@pytest.mark.parametrize("ld,offset", [(1008, 0), (1008, 8), (1001, 0), (1000, 1)])
def test_backward_strides_and_alignment(ld, offset):
    device()
    _, h, w, dy, dh = data(50, 1000, torch.bfloat16, 7)
    rstd = rstd_of(h)
    check_backward(backward(dy, h, w, rstd, dh, ld, offset), dy, h, w, rstd, dh)


@pytest.mark.parametrize("cols", [100, 1024, 4096, 20000])
@pytest.mark.parametrize("into", ["dy", "dh"])
def test_backward_in_place(into, cols):
    device()
    _, h, w, dy, dh = data(90, cols, torch.bfloat16, 8)
    rstd = rstd_of(h)
    check_backward(backward(dy, h, w, rstd, dh, in_place=into), dy, h, w, rstd, dh)


def test_backward_without_rows():
    dev = device()
    w = torch.ones(300, dtype=torch.bfloat16, device=dev)
    dw = torch.full((300,), 7.0, dtype=torch.bfloat16, device=dev)
    none = torch.empty(0, 300, dtype=torch.bfloat16, device=dev)
    zr.zr_rmsnorm_backward(none, none, w, torch.empty(0, device=dev), none.clone(), dw, zr.rmsnorm_workspace(300))
    assert bool((dw == 0).all())


def test_backward_against_differences():
    """dx and dweight against central differences of the 64-bit forward formula.  The loss
    is a sum of y * dy: a difference with step 1e-4 is off by O(1e-8) of values near 1,
    far below the 16-bit rounding that check_backward's bound holds."""
    device()
    rows, cols, eps, d = 2, 96, 1e-5, 1e-4
    _, h, w, dy, _ = data(rows, cols, torch.float16, 9)
    got_dx, got_dw = backward(dy, h, w, rstd_of(h))
    hd, wd, dyd = h.double().cpu(), w.double().cpu(), dy.double().cpu()

    def loss(hh, ww):
        return (hh / torch.sqrt(hh.pow(2).mean(1, keepdim=True) + eps) * ww * dyd).sum()

    for i in range(rows):
        for j in range(0, cols, 5):
            e = torch.zeros_like(hd)
            e[i, j] = d
            want = (loss(hd + e, wd) - loss(hd - e, wd)) / (2 * d)
            assert abs(float(got_dx[i, j]) - want) <= HALF[torch.float16] * abs(want) + 1e-5
    for j in range(cols):
        e = torch.zeros_like(wd)
        e[j] = d
        want = (loss(hd, wd + e) - loss(hd, wd - e)) / (2 * d)
        assert abs(float(got_dw[j]) - want) <= HALF[torch.float16] * abs(want) + 1e-5


def test_wide_offsets():
    """Row offsets past 2^31 elements."""
    dev = device()
    ld = (1 << 30) + 8
    big = torch.zeros(2 * ld + 256, dtype=torch.bfloat16, device=dev)
    x, _, w, dy, _ = data(3, 256, torch.bfloat16, 10)
    v = big.as_strided((3, 256), (ld, 1), 0)
    v.copy_(x)
    q, s = zr.fp8_matrix(3, 256)
    y = torch.empty(3, 256, dtype=torch.bfloat16, device=dev)
    rstd = torch.empty(3, device=dev)
    zr.zr_rmsnorm_fp8(v, w, y, q, s, rstd=rstd)
    check_forward({"h": None, "y": y, "q": q, "s": s.view(torch.uint8), "rstd": rstd}, x, w)
    dx, dw = torch.empty_like(y), torch.empty_like(w)
    zr.zr_rmsnorm_backward(dy, v, w, rstd, dx, dw, zr.rmsnorm_workspace(256))
    check_backward((dx, dw), dy, x, w, rstd)


@pytest.mark.parametrize("rows,cols", [(700, 1000), (40, 20000), (90, 4096)])
def test_capped_grid(monkeypatch, rows, cols):
    """Results are the same bits whatever the grid."""
    device()
    x, res, w, dy, dh = data(rows, cols, torch.bfloat16, 11)
    rstd = rstd_of(x)

    def run():
        out = forward(x, w, res)
        return [out[k].contiguous().view(torch.uint8).clone() for k in ("h", "y", "q", "s")] + \
               [out["rstd"].clone()] + [t.clone() for t in backward(dy, x, w, rstd, dh)]

    full = run()
    for cap in ("8", "24"):
        monkeypatch.setenv("ZR_MAX_GRID", cap)
        assert all(torch.equal(a, b) for a, b in zip(run(), full)), cap
