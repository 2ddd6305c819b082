"""zr_qk_norm_rope and zr_qk_norm_rope_backward on the GPU against the formulas in 64 bits.

Tolerances, with U = 2^-24 (half a step of fp32).  A lane adds at most 16 squares, then 6
additions join the lanes: the sum is off by 22 U relative, rstd by half of that and 4
operations: 15 U.  A cosine or sine: the part of a turn, at most 1/2, is rounded to fp32
(2 pi / 2 U = 3.2 U of angle), sincospi is right to 2 units in the last place (4 U), the fp64
angle to 2^-52 of itself (8 U at an angle of 2^31): 16 U in all.  An output pair then is
off by at most (|y_a| + |y_b|) times rstd's 15 U, two products' 2 U, the turn's 16 U and two
operations' 2 U: 40 U with some room; then it is rounded once to the type, half a step.
Backward: with G = (|dy_a| + |dy_b|) |w| and A = mean of G |x| * rstd^2, the turned gradient
times the weight is off by 20 U G, the mean by A times 20 + 24 (its sum) + 30 (rstd^2) + 3
U, and dx by rstd (G + |x| A) 100 U.  A weight gradient's term g xh is off by 38 U of
(|dy_a| + |dy_b|) |xh|, and its sum over `rows` terms takes at most rows / 32 + 128 additions
one after another.
"""
import itertools

import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from fp8_util import HALF, TINY
from gpu_util import device

pytestmark = pytest.mark.gpu
BF, FP16 = torch.bfloat16, torch.float16
U = 2.0 ** -24
inf, nan = float("inf"), float("nan")


def frequencies(rot, base=1e4):
    return (base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(1, rot))).float()


def pair_index(rot, interleaved):
    j = torch.arange(rot // 2, device="cuda")
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def angles(positions, rope):
    """[tokens, 1, pairs] in 64 bits."""
    pos = positions.view(-1, positions.shape[-1]).double()
    axis = torch.tensor(list(rope._axis)[:rope.inv_freq.numel()], device="cuda") if rope._axis is not None else \
        torch.zeros(rope.inv_freq.numel(), dtype=torch.int64, device="cuda")
    return (pos[axis.long()].t() * rope.inv_freq.double())[:, None]


def turn(y, angle, rot, interleaved, back=False):
    a, b = pair_index(rot, interleaved)
    c, s = torch.cos(angle), torch.sin(angle) * (-1 if back else 1)
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def pair_sum(y, rot, interleaved):
    """|y_a| + |y_b| at both elements of a pair, |y| elsewhere."""
    a, b = pair_index(rot, interleaved)
    out = y.abs().clone()
    out[..., a] = out[..., b] = y[..., a].abs() + y[..., b].abs()
    return out


def forward(x, w, angle, rot, interleaved, eps):
    x = x.double()
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.double() if w is not None else x
    return turn(y, angle, rot, interleaved), 40 * U * pair_sum(y, rot, interleaved)


def backward(dy, x, w, angle, rot, interleaved, eps):
    """dx, dw and their bounds without the output's rounding."""
    dy = dy.double()
    g, size = turn(dy, angle, rot, interleaved, back=True), pair_sum(dy, rot, interleaved)
    if w is None:
        return g, None, 40 * U * size, None
    x, w = x.double(), w.double()
    rstd = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    gw, big = g * w, size * w.abs()
    dx = rstd * (gw - x * rstd ** 2 * (gw * x).mean(-1, keepdim=True))
    along = (big * x.abs()).mean(-1, keepdim=True) * rstd ** 2
    rows = x.shape[0] * x.shape[1]
    dw = (g * x * rstd).sum((0, 1))
    return dx, dw, rstd * (big + x.abs() * along) * 100 * U, (size * x.abs() * rstd).sum((0, 1)) * (38 + rows / 32 + 128) * U


def near(got, want, bound, what):
    t = got.dtype
    want = want.to(t).double() if not torch.isfinite(want).all() else want
    off = (got.double() - want).abs()
    limit = bound + HALF[t] * (want.abs() + bound) + TINY[t]
    bad = ~(off <= limit)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / limit).max()):.3g} of the bound"


def rows(t, h, d, dtype, seed, layout="heads", size=1.0):
    """[t, h, d] of random values as a view of `layout`, with the buffer that holds it: plain heads, heads of a wider
    row at an odd element, or heads before tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(t, h, d, generator=g, device="cuda") * torch.exp(torch.randn(t, 1, 1, generator=g, device="cuda") * 0.5)
         * size).to(dtype)
    if layout == "heads":
        raw = torch.full((t * h * d + 64,), 9.0, dtype=dtype, device="cuda")
        v = raw[:t * h * d].view(t, h, d)
    elif layout == "row":
        width = (h + 3) * d + 5
        raw = torch.full((t * width + 64,), 9.0, dtype=dtype, device="cuda")
        v = raw.as_strided((t, h, d), (width, d, 1), 3)
    else:
        raw = torch.full((t * h * d + 64,), 9.0, dtype=dtype, device="cuda")
        v = raw[:t * h * d].view(h, t, d).transpose(0, 1)
    v.copy_(x)
    return v, raw


def blank(v, raw):
    """The same view of a buffer of 9s."""
    new = torch.full_like(raw, 9.0)
    return new.as_strided(v.shape, v.stride(), v.storage_offset()), new


def untouched(v, raw):
    keep = torch.ones_like(raw, dtype=torch.bool)
    keep.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
    return bool((raw[keep] == 9.0).all())


def case(t, hq, hk, d, rot, dtype, interleaved=False, axes=1, far=0, layout="heads", seed=0, normed=(True, True), base=1e4):
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    half = rot // 2
    axis = torch.randint(0, axes, (half,), generator=g, device="cuda").tolist() if axes > 1 else None
    if axis:
        axis[-1] = axes - 1
    c = dict(rope=zr.rope(frequencies(rot, base), interleaved=interleaved, pair_axis=axis), rot=rot, interleaved=interleaved)
    pos = torch.randint(0, max(1, far or 4096), (axes, t), generator=g, device="cuda")
    c["positions"] = pos if axes > 1 else pos[0]
    c["q"], c["q_raw"] = rows(t, hq, d, dtype, seed + 1, layout)
    c["k"], c["k_raw"] = rows(t, hk, d, dtype, seed + 2, layout)
    c["wq"], c["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) if on else None for on in normed)
    c["angle"] = angles(c["positions"], c["rope"])
    return c


def check_forward(c, eps=1e-5, in_place=False):
    want = [forward(c[x], c["w" + x], c["angle"], c["rot"], c["interleaved"], eps) for x in "qk"]
    out = [(c[x], c[x + "_raw"]) if in_place else blank(c[x], c[x + "_raw"]) for x in "qk"]
    zr.zr_qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["rope"], out[0][0], out[1][0], eps=eps)
    for (v, raw), (y, bound), name in zip(out, want, "qk"):
        near(v, y, bound, name)
        assert untouched(v, raw)
    return [v for v, _ in out]


def check_backward(c, eps=1e-5, in_place=None):
    grads = [rows(*c[x].shape, c[x].dtype, 77 + i, "heads", 0.3) for i, x in enumerate("qk")]
    want = [backward(grads[i][0], c[x], c["w" + x], c["angle"], c["rot"], c["interleaved"], eps) for i, x in enumerate("qk")]
    out = [grads[i] if in_place == "dy" else (c[x], c[x + "_raw"]) if in_place == "x" else blank(c[x], c[x + "_raw"])
           for i, x in enumerate("qk")]
    d = c["q"].shape[2]
    dw = [torch.full((d + 9,), 9.0, dtype=c["q"].dtype, device="cuda") for _ in "qk"]
    ws = torch.full((zr.ZR_QK_PARTIALS, d), nan, device="cuda")
    zr.zr_qk_norm_rope_backward(grads[0][0], grads[1][0], c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["rope"], out[0][0],
                                out[1][0], dw[0][:d] if c["wq"] is not None else None, dw[1][:d] if c["wk"] is not None else None,
                                ws, eps=eps)
    for i, name in enumerate("qk"):
        dx, dwant, bx, bw = want[i]
        near(out[i][0], dx, bx, "d" + name)
        assert untouched(*out[i])
        assert bool((dw[i][d:] == 9).all())
        if dwant is not None:
            near(dw[i][:d], dwant, bw, f"d{name}_weight")
    return [v for v, _ in out] + [x[:d] for x in dw]


DIMS = [(128, 128), (128, 64), (128, 32), (64, 64), (96, 96), (80, 80), (80, 20), (72, 72), (88, 40), (256, 256), (256, 64),
        (512, 512), (512, 128), (200, 200), (40, 40), (16, 16), (2, 2), (6, 4), (7, 6), (1, 0), (33, 18), (127, 126), (129, 128),
        (511, 510), (300, 298), (128, 0), (50, 50), (130, 130), (512, 510), (509, 0), (127, 8), (511, 500), (66, 66), (80, 18),
        (300, 2), (512, 6), (24, 8), (23, 16), (9, 8), (8, 6), (17, 16), (31, 14), (260, 256), (130, 0), (5, 0), (3, 2)]


@pytest.mark.parametrize("dtype", [BF, FP16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", DIMS)
def test_head_sizes(d, rot, interleaved, dtype):
    device()
    for t in (13, 2100):  # few steps and many (over 4096) have kernels of their own
        c = case(t, 5, 3, d, rot, dtype, interleaved, seed=d + rot)
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("layout", ["heads", "row", "before"])
@pytest.mark.parametrize("t,hq,hk", [(1, 1, 1), (1, 32, 8), (3, 40, 40), (7, 9, 1), (257, 32, 8), (1000, 4, 4), (2, 64, 2), (5, 17, 16)])
def test_tokens_heads_and_strides(t, hq, hk, layout):
    device()
    for dtype, d, rot in ((BF, 128, 128), (FP16, 72, 72), (BF, 66, 22)):
        c = case(t, hq, hk, d, rot, dtype, layout=layout, seed=t)
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(axes, interleaved):
    device()
    for d, rot in ((96, 96), (128, 96), (33, 18)):
        c = case(130, 6, 2, d, rot, BF, interleaved, axes=axes, seed=axes)
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("far", [131_072, 1 << 20, 1 << 31])
def test_far_positions(far):
    """The angle keeps its place in the turn."""
    device()
    c = case(300, 4, 2, 128, 128, FP16, far=far, base=1e6)
    c["positions"][:3] = torch.tensor([far - 1, -far, 0], device="cuda")
    c["angle"] = angles(c["positions"], c["rope"])
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("normed", [(False, False), (True, False), (False, True)])
def test_without_norm(normed):
    """Turned only; elements past the turned part keep their bits, whatever they are."""
    device()
    for d, rot in ((128, 64), (72, 40), (33, 18)):
        c = case(50, 6, 3, d, rot, BF, normed=normed)
        check_forward(c)
        check_backward(c)
    c = case(20, 4, 4, 128, 64, BF, normed=(False, False))
    g = torch.Generator(device="cuda").manual_seed(1)
    c["q"][..., 64:] = torch.randint(-2 ** 15, 2 ** 15 - 1, (20, 4, 64), generator=g, device="cuda").to(torch.int16).view(BF)
    q, k = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    zr.zr_qk_norm_rope(c["q"], c["k"], None, None, c["positions"], c["rope"], q, k)
    want = c["q"][..., 64:].contiguous()
    same = (q[..., 64:].contiguous().view(torch.int16) == want.view(torch.int16)) | (want.isnan() & q[..., 64:].isnan())
    assert bool(same.all())


@pytest.mark.parametrize("d,rot", [(128, 128), (72, 72), (33, 18), (300, 298)])
def test_in_place(d, rot):
    device()
    for layout in ("heads", "row", "before"):
        args = (70, 6, 2, d, rot, FP16)
        plain = check_forward(case(*args, layout=layout))
        for a, b in zip(plain, check_forward(case(*args, layout=layout), in_place=True)):
            assert torch.equal(a, b)
        plain = check_backward(case(*args, layout=layout))
        for how in ("dy", "x"):
            for a, b in zip(plain, check_backward(case(*args, layout=layout), in_place=how)):
                assert torch.equal(a, b)


def test_queries_and_keys_of_one_fused_row():
    """Queries and keys turned where they lie, between values that stay as they are."""
    device()
    t, hq, hk, d = 41, 8, 2, 64
    c = case(t, hq, hk, d, d, BF)
    fused = torch.full((t, (hq + 2 * hk) * d), 3.0, dtype=BF, device="cuda")
    q, k = fused[:, :hq * d].view(t, hq, d), fused[:, hq * d:(hq + hk) * d].view(t, hk, d)
    q.copy_(c["q"])
    k.copy_(c["k"])
    want = check_forward(c)
    zr.zr_qk_norm_rope(q, k, c["wq"], c["wk"], c["positions"], c["rope"], q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and bool((fused[:, (hq + hk) * d:] == 3).all())
    # one token: a row of heads without a token distance
    zr.zr_qk_norm_rope(q[:1], k[:1], c["wq"], c["wk"], c["positions"][:1], c["rope"], q[:1], k[:1])


def test_one_tensor_alone():
    device()
    c = case(30, 6, 3, 128, 128, BF)
    both = check_forward(c)
    q, k = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    zr.zr_qk_norm_rope(c["q"], None, c["wq"], None, c["positions"], c["rope"], q, None)
    zr.zr_qk_norm_rope(None, c["k"], None, c["wk"], c["positions"], c["rope"], None, k)
    assert torch.equal(q, both[0]) and torch.equal(k, both[1])
    dq, dwq, ws = torch.empty_like(q), torch.empty(128, dtype=BF, device="cuda"), zr.qk_norm_workspace(128)
    zr.zr_qk_norm_rope_backward(q, None, c["q"], None, c["wq"], None, c["positions"], c["rope"], dq, None, dwq, None, ws)
    dx, dw, bx, bw = backward(q, c["q"], c["wq"], c["angle"], 128, False, 1e-5)
    near(dq, dx, bx, "dq")
    near(dwq, dw, bw, "dq_weight")


def test_no_tokens_and_no_heads():
    device()
    c = case(4, 2, 2, 64, 64, BF)
    e = lambda t, h: torch.empty(t, h, 64, dtype=BF, device="cuda")  # noqa: E731
    dwq, dwk = (torch.full((64,), 5.0, dtype=BF, device="cuda") for _ in "qk")
    ws = zr.qk_norm_workspace(64)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    zr.zr_qk_norm_rope(e(0, 2), e(0, 2), c["wq"], c["wk"], none, c["rope"], e(0, 2), e(0, 2))
    zr.zr_qk_norm_rope_backward(e(0, 2), e(0, 2), e(0, 2), e(0, 2), c["wq"], c["wk"], none, c["rope"], e(0, 2), e(0, 2), dwq, dwk, ws)
    assert not dwq.any() and not dwk.any()
    dwk.fill_(5.0)
    zr.zr_qk_norm_rope_backward(c["q"], e(4, 0), c["q"], e(4, 0), c["wq"], c["wk"], c["positions"], c["rope"], e(4, 2), e(4, 0), dwq,
                                dwk, ws)
    assert dwq.any() and not dwk.any()


def test_infinities_stay_in_their_row():
    device()
    c = case(9, 4, 2, 128, 128, BF)
    clean = check_forward(c)
    for at, v in (((2, 1), inf), ((4, 3), nan)):
        c["q"][at][5] = v
    q, k = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    zr.zr_qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["rope"], q, k)
    assert bool(q[4, 3].isnan().all()) and bool(q[2, 1, 5].isnan()) and bool(q[2, 1, 69].isnan())
    rest = torch.ones(9, 4, dtype=torch.bool, device="cuda")
    rest[2, 1] = rest[4, 3] = False
    assert torch.equal(q[rest], clean[0][rest]) and torch.equal(k, clean[1])
    zero = torch.zeros(3, 2, 128, dtype=BF, device="cuda")  # rows of zeros: eps keeps them
    out = torch.empty_like(zero)
    zr.zr_qk_norm_rope(zero, None, c["wq"], None, c["positions"][:3], c["rope"], out, None)
    assert not out.any()


@pytest.mark.parametrize("d,rot", [(128, 128), (66, 66), (33, 18)])
def test_gradients_of_rows_with_infinities(d, rot):
    """An infinity in a row of x makes its gradients NaN and the weight's at its own column (the others
    get nothing of the row: its rstd is 0); a NaN makes all of the weight's NaN.  An infinite gradient makes
    the row's NaN.  The other rows are as without them."""
    device()
    c = case(12, 6, 2, d, rot, BF)
    dy = [torch.randn(c[x].shape, device="cuda").to(BF) for x in "qk"]
    clean = backward_of(c, dy)
    c["q"][7, 5] = 0.0
    zeroed = backward_of(c, dy)[2]
    keep = torch.ones(12, 6, dtype=torch.bool, device="cuda")
    keep[7, 5] = False
    for value in (inf, -inf, nan):
        c["q"][7, 5] = 1.0
        c["q"][7, 5, 3] = value
        dq, dk, dwq, dwk = backward_of(c, dy)
        assert bool(dq[~keep].isnan().all()) and torch.equal(dq[keep], clean[0][keep])
        assert torch.equal(dk, clean[1]) and torch.equal(dwk, clean[3])
        other = torch.arange(d, device="cuda") != 3
        assert bool(dwq[3].isnan())
        assert bool(dwq.isnan().all()) if value != value else torch.equal(dwq[other], zeroed[other])
    c["q"][7, 5] = 1.0
    dy[0][7, 5, 0] = inf
    dq, dk, _, dwk = backward_of(c, dy)
    assert not bool(dq[~keep].isfinite().any()) and torch.equal(dq[keep], clean[0][keep])
    assert torch.equal(dk, clean[1]) and torch.equal(dwk, clean[3])


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-31, 1e-6, 3.0])
def test_eps(eps):
    """Both ways of the reciprocal root.  Values of 1e-12 (squares of 1e-24) and of 1: the
    first are all eps at 1e-6, and none of it at 1e-31."""
    device()
    for d, rot in ((128, 128), (33, 18)):
        c = case(40, 5, 3, d, rot, BF)
        c["q"][::2] *= 1e-12
        check_forward(c, eps=eps)
        check_backward(c, eps=eps)


def test_rows_of_zeros_without_eps():
    """0 / 0 in their own rows alone; their gradient is NaN, as the formula's."""
    device()
    c = case(9, 5, 3, 128, 128, BF)
    clean = check_forward(c, eps=0.0)
    c["q"][4, 2] = 0.0
    q, k = torch.empty_like(clean[0]), torch.empty_like(clean[1])
    zr.zr_qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["rope"], q, k, eps=0.0)
    rest = torch.ones(9, 5, dtype=torch.bool, device="cuda")
    rest[4, 2] = False
    assert bool(q[4, 2].isnan().all()) and torch.equal(q[rest], clean[0][rest]) and torch.equal(k, clean[1])


@pytest.mark.parametrize("d,rot", [(128, 128), (66, 66), (33, 18)])
def test_rows_past_the_range_of_their_squares(d, rot):
    """Magnitudes of 1e20 and more: rstd 0, and with it the outputs and every gradient; the other
    rows are as without them."""
    device()
    c = case(12, 6, 2, d, rot, BF)
    clean = check_forward(c)
    at = [(1, 0), (7, 5), (11, 3)]
    dy = [torch.randn(x.shape, device="cuda").to(BF) for x in clean]
    run = lambda: backward_of(c, dy)  # noqa: E731
    for token, head in at:
        c["q"][token, head] = 0.0
    dq0, _, dwq0, _ = run()
    for i, (token, head) in enumerate(at):
        c["q"][token, head] = torch.tensor([1e20, -1e30, 3e38][i], device="cuda").to(BF)
    q, k = torch.empty_like(clean[0]), torch.empty_like(clean[1])
    zr.zr_qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["rope"], q, k)
    dq, _, dwq, _ = run()
    keep = torch.ones(12, 6, dtype=torch.bool, device="cuda")
    for token, head in at:
        keep[token, head] = False
    assert not q[~keep].any() and torch.equal(q[keep], clean[0][keep])
    assert not dq[~keep].any() and torch.equal(dq[keep], dq0[keep])
    assert torch.equal(dwq, dwq0)


def backward_of(c, dy, eps=1e-5):
    d = c["q"].shape[2]
    out = [torch.empty_like(x) for x in dy] + [torch.empty(d, dtype=BF, device="cuda") for _ in "qk"]
    zr.zr_qk_norm_rope_backward(*dy, c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["rope"], *out, zr.qk_norm_workspace(d), eps=eps)
    return out


@pytest.mark.parametrize("d,rot", [(128, 128), (72, 72), (33, 18)])
def test_same_bits_on_any_grid(d, rot, monkeypatch):
    device()
    for t in (40, 300, 3000):
        c = case(t, 12, 4, d, rot, BF)
        one = check_forward(c) + check_backward(c)
        for cap in ("8", "24"):
            monkeypatch.setenv("ZR_MAX_GRID", cap)
            for a, b in zip(one, check_forward(c) + check_backward(c)):
                assert torch.equal(a, b)
        monkeypatch.delenv("ZR_MAX_GRID")


def test_gradient_against_differences():
    """dx . u and dw . u against central differences of the forward formula in 64 bits along
    random directions u (step 1e-5: the differences' own error is near 1e-9 of the loss); the
    bound is what the tolerances of dx and dw allow along u."""
    device()
    for d, rot, interleaved in ((128, 128, False), (72, 40, True)):
        c = case(11, 3, 2, d, rot, FP16, interleaved)
        g = torch.Generator(device="cuda").manual_seed(3)
        dy = torch.randn(11, 3, d, generator=g, device="cuda").to(FP16)
        dx, dw = torch.empty_like(dy), torch.empty(d, dtype=FP16, device="cuda")
        zr.zr_qk_norm_rope_backward(dy, None, c["q"], None, c["wq"], None, c["positions"], c["rope"], dx, None, dw, None,
                                    zr.qk_norm_workspace(d))
        x, w = c["q"].double(), c["wq"].double()
        loss = lambda x, w: float((forward(x, w, c["angle"], rot, interleaved, 1e-5)[0] * dy.double()).sum())  # noqa: E731
        _, _, bx, bw = backward(dy, x, w, c["angle"], rot, interleaved, 1e-5)
        for _ in range(5):
            u, uw = (torch.randn(s.shape, generator=g, device="cuda", dtype=torch.float64) for s in (x, w))
            h = 1e-5
            got, want = float((dx.double() * u).sum()), (loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h)
            room = float(((bx + HALF[FP16] * dx.double().abs() + TINY[FP16]) * u.abs()).sum())
            assert abs(got - want) <= room + 1e-6 * abs(want) + 1e-6
            got, want = float((dw.double() * uw).sum()), (loss(x, w + h * uw) - loss(x, w - h * uw)) / (2 * h)
            room = float(((bw + HALF[FP16] * dw.double().abs() + TINY[FP16]) * uw.abs()).sum())
            assert abs(got - want) <= room + 1e-6 * abs(want) + 1e-6


def test_past_32_bits():
    """Tokens whose rows lie past 2^32 bytes and 2^31 elements from the first."""
    device()
    t, h, d, width = 3, 2, 128, (1 << 30) + 8
    c = case(t, h, h, d, d, BF)
    raw = torch.empty(2 * width + 4 * d, dtype=BF, device="cuda")
    q = raw.as_strided((t, h, d), (width, d, 1), 0)
    q.copy_(c["q"])
    want = check_forward(c)[0]
    zr.zr_qk_norm_rope(q, None, c["wq"], None, c["positions"], c["rope"], q, None)
    assert torch.equal(q, want)
    dq, ws = torch.empty_like(want), zr.qk_norm_workspace(d)
    q.copy_(c["q"])
    dw = [torch.empty(d, dtype=BF, device="cuda") for _ in range(2)]
    zr.zr_qk_norm_rope_backward(want, None, c["q"], None, c["wq"], None, c["positions"], c["rope"], dq, None, dw[0], None, ws)
    zr.zr_qk_norm_rope_backward(want, None, q, None, c["wq"], None, c["positions"], c["rope"], q, None, dw[1], None, ws)
    assert torch.equal(q, dq) and torch.equal(*dw)


@pytest.mark.parametrize("seed", range(12))
def test_random_cases(seed):
    import random
    device()
    r = random.Random(seed)
    for _ in range(6):
        d = r.choice([r.randint(1, 512), 8 * r.randint(1, 64), 128, 64])
        rot = r.choice([d // 2 * 2, r.randint(0, d // 2) * 2])
        t, hq = r.choice([1, 2, r.randint(1, 600)]), r.randint(1, 40)
        c = case(t, hq, r.randint(1, hq), d, rot, r.choice([BF, FP16]), r.random() < 0.5, r.randint(1, 4) if rot > 6 else 1,
                 r.choice([0, 100_000]), r.choice(["heads", "row", "before"]), seed, (r.random() < 0.8, r.random() < 0.8))
        check_forward(c, in_place=False)
        check_backward(c)
