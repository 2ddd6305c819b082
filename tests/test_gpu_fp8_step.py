"""The 8-bit operators together, as a training step and a replayed graph use them, with
the calls of zr.h around them: a linear layer behind a norm, from the gathered
parameter shard to the AdamW update of the gradient's slice."""
import threading

import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from fp8_util import E4M3, E5M2, HALF, groups, values
from gpu_util import device

pytestmark = pytest.mark.gpu


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def layer(tokens, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return r(tokens, k), r(tokens, k), (1 + 0.1 * r(k)).to(torch.bfloat16), (0.05 * r(n, k)), r(tokens, n)


class Step:
    """x, res -> h, norm, codes -> y = norm W^T; dy -> dx, dW and the norm's gradients."""

    def __init__(self, x, res, w_norm, w, dy):
        (t, k), n = x.shape, w.shape[0]
        self.x, self.res, self.w_norm, self.w, self.dy = x, res, w_norm, w, dy
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.h, self.norm, self.rstd = bf(t, k), bf(t, k), torch.empty(t, device="cuda")
        self.q, self.s = zr.fp8_matrix(t, k)
        self.wq, self.ws = zr.fp8_matrix(n, k, block_rows=128)
        self.wt, self.wts = zr.fp8_matrix(k, n, block_rows=128)
        self.y = bf(t, n)
        self.dq, self.ds = zr.fp8_matrix(t, n, E5M2)
        self.dqt, self.dst = zr.fp8_matrix(n, t, E5M2)
        self.nqt, self.nst = zr.fp8_matrix(k, t)
        self.dnorm, self.dw, self.dx, self.dw_norm = bf(t, k), bf(n * k), bf(t, k), bf(k)
        self.workspace = zr.rmsnorm_workspace(k)

    def run(self, stream=None):
        kw = dict(stream=stream)
        zr.zr_quantize_fp8(self.w, self.wq, self.ws, self.wt, self.wts, block_rows=128, **kw)
        zr.zr_rmsnorm_fp8(self.x, self.w_norm, self.norm, self.q, self.s, residual=self.res, h=self.h, rstd=self.rstd, **kw)
        zr.zr_matmul_fp8(self.q, self.s, self.wq, self.ws, self.y, b_block_rows=128, **kw)
        zr.zr_quantize_fp8(self.dy, self.dq, self.ds, self.dqt, self.dst, **kw)
        zr.zr_quantize_fp8(self.norm, qt=self.nqt, scales_t=self.nst, **kw)
        zr.zr_matmul_fp8(self.dq, self.ds, self.wt, self.wts, self.dnorm, b_block_rows=128, **kw)
        zr.zr_matmul_fp8(self.dqt, self.dst, self.nqt, self.nst, self.dw.view(self.w.shape), **kw)
        zr.zr_rmsnorm_backward(self.dnorm, self.h, self.w_norm, self.rstd, self.dx, self.dw_norm, self.workspace, dh=self.dnorm, **kw)

    def outputs(self):
        return [t.clone() for t in (self.y, self.dw, self.dx, self.dw_norm, self.h, self.rstd)]


@pytest.mark.parametrize("tokens,n,k", [(200, 512, 1024), (131, 384, 640), (1000, 1536, 512)])
def test_layer_gradients(tokens, n, k):
    """Against autograd of the same layer in 64 bits.  A code is off by at most 2^-4 (e4m3) or
    2^-3 (e5m2) of its value, a product of two by their sum; errors of unlike sign add up as
    their root mean square, at most 1 / sqrt(3) of the largest: the relative distance of a
    product stays below (2^-4 + 2^-4) / sqrt(3) (e4m3 twice) or (2^-4 + 2^-3) / sqrt(3)."""
    device()
    x, res, w_norm, w, dy = layer(tokens, n, k, tokens)
    s = Step(x, res, w_norm, w, dy)
    s.run()
    h = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(s.h, h)
    hd, wn, wd = (t.double().requires_grad_() for t in (h, w_norm, w))
    norm = hd / torch.sqrt(hd.pow(2).mean(1, keepdim=True) + 1e-5) * wn
    y = norm @ wd.t()
    (y * dy.double()).sum().backward()
    near, far = 2.0 ** -3 / 3 ** 0.5, (2.0 ** -4 + 2.0 ** -3) / 3 ** 0.5
    assert rel(s.y, y.detach()) < near
    assert rel(s.dw.view(n, k), wd.grad) < far
    dnorm = dy.double() @ wd.detach()
    assert rel(s.dnorm, dnorm) < far
    assert rel(s.dx, hd.grad + dnorm) < far
    assert rel(s.dw_norm, wn.grad) < far


def test_gathered_codes_are_the_products_operand():
    """Shards of a flat parameter buffer, quantized as they lie, gathered by concatenation: the
    codes and scales of a tensor whose rows are whole groups are its rows' codes and scales, and
    the product takes them in place; dW goes to the flat gradient buffer, whose slice is reduced
    and stepped."""
    dev = device()
    n_d, shapes = 4, [(384, 512), (256, 768), (100,)]
    numels = [384 * 512, 256 * 768, 100]
    lay = zr.zr_layout_create(numels, n_d, 1000)
    info = zr.zr_layout_query(lay)
    S = info["shard"]
    assert S % 128 == 0
    g = torch.Generator(device="cuda").manual_seed(3)
    w = [(0.05 * torch.randn(x, generator=g, device="cuda")).to(torch.bfloat16) for x in numels[:2]]
    codes = torch.empty(info["psi_pad"], dtype=E4M3, device=dev)
    scales = torch.empty(info["psi_pad"] // 128, dtype=torch.float8_e8m0fnu, device=dev)
    for r in range(n_d):
        b, e = zr.zr_layout_rank_range(lay, r)
        shard = torch.empty(S, dtype=torch.bfloat16, device=dev)
        zr.zr_pack(lay, w + [None], shard, b, e)
        zr.zr_quantize_fp8(shard, codes[b:e], scales[b // 128:e // 128])
    grads = torch.zeros(info["psi_pad"], dtype=torch.bfloat16, device=dev)
    for t, shape in enumerate(shapes[:2]):
        _, off = zr.zr_layout_tensor(lay, t)
        q = codes[off:off + numels[t]].view(shape)
        s = scales[off // 128:(off + numels[t]) // 128].view(shape[0], groups(shape[1]))
        x = torch.randn(50, shape[1], generator=g, device="cuda").to(torch.bfloat16)
        xq, xs = zr.fp8_matrix(50, shape[1])
        zr.zr_quantize_fp8(x, xq, xs)
        y = torch.empty(50, shape[0], dtype=torch.bfloat16, device=dev)
        zr.zr_matmul_fp8(xq, xs, q, s, y, b_block_rows=1)
        want = values(xq, xs.view(torch.uint8)) @ values(q, s.view(torch.uint8)).t()
        assert rel(y, want) < HALF[torch.bfloat16]
        # a gradient of y's size, straight into the tensor's piece of the flat buffer, twice
        dqt, dst = zr.fp8_matrix(shape[0], 50)
        xt, xts = zr.fp8_matrix(shape[1], 50)
        zr.zr_quantize_fp8(y, qt=dqt, scales_t=dst)
        zr.zr_quantize_fp8(x, qt=xt, scales_t=xts)
        piece = grads[off:off + numels[t]].view(shape)
        want = values(dqt, dst.view(torch.uint8)) @ values(xt, xts.view(torch.uint8)).t()
        zr.zr_matmul_fp8(dqt, dst, xt, xts, piece)
        assert rel(piece, want) < HALF[torch.bfloat16]
        zr.zr_matmul_fp8(dqt, dst, xt, xts, piece, accumulate=True)
        assert rel(piece, 2 * want) < 2 * HALF[torch.bfloat16]
    b, e = zr.zr_layout_rank_range(lay, 1)
    mean, master, m, v = torch.empty(S, dtype=torch.bfloat16, device=dev), *(torch.zeros(S, device=dev) for _ in range(3))
    zr.zr_reduce_slice([grads[b:e], grads[b:e]], mean)
    assert torch.equal(mean, grads[b:e])
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    zr.zr_adamw_step(mean, master, m, v, None, **hp)
    moved = mean != 0
    assert bool((master[moved].sign() == -mean[moved].float().sign()).all())


def test_captured_step_replays():
    """The step as one graph of zr.h, replayed between eager runs on other data: every replay
    is the eager result, and a second graph of the same calls with a workspace of its own does not
    disturb the first."""
    device()
    a, b = layer(300, 512, 640, 1), layer(300, 512, 640, 2)
    eager = Step(*a)
    eager.run()
    want_a = eager.outputs()
    other = Step(*b)
    other.run()
    want_b = other.outputs()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, steps = [], [Step(*a), Step(*b)]
    with torch.cuda.stream(stream):
        for s in steps:
            zr.zr_graph_capture_begin(stream)
            s.run(stream)
            graphs.append(zr.zr_graph_capture_end(stream))
    assert zr.zr_graph_info(graphs[0])[0] == 9  # the norm's backward pass is two kernels
    for turn in range(4):
        for gr in graphs:
            zr.zr_graph_launch(gr, stream)
        stream.synchronize()
        for s, want in zip(steps, (want_a, want_b)):
            assert all(torch.equal(x, y) for x, y in zip(s.outputs(), want)), turn
        # new inputs in place: the replay follows them
        steps[0].x.copy_(b[0] if turn % 2 == 0 else layer(300, 512, 640, 1)[0])
        eager.x.copy_(steps[0].x)
        eager.run()
        torch.cuda.synchronize()
        want_a = eager.outputs()


def test_streams_and_threads():
    """The same calls on several streams and from several threads at once, each with buffers
    of its own, give what they give alone."""
    device()
    data = [layer(257, 384, 512, 10 + i) for i in range(4)]
    want = []
    for d in data:
        s = Step(*d)
        s.run()
        want.append(s.outputs())
    torch.cuda.synchronize()
    steps, streams = [Step(*d) for d in data], [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    errors = []

    def work(s, st):
        try:
            with torch.cuda.stream(st):
                for _ in range(5):
                    s.run()  # on torch's current stream
            st.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, streams)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for s, w in zip(steps, want):
        assert all(torch.equal(x, y) for x, y in zip(s.outputs(), w))


def test_capture_refuses_what_eager_refuses():
    """A refused call inside a capture records nothing and says why."""
    device()
    stream = torch.cuda.Stream()
    q, s = zr.fp8_matrix(8, 256)
    x = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        zr.zr_graph_capture_begin(stream)
        with pytest.raises(zr.ZRError):
            zr.zr_quantize_fp8(x, q, s, block_rows=64, stream=stream)
        zr.zr_quantize_fp8(x, q, s, stream=stream)
        gr = zr.zr_graph_capture_end(stream)
    assert zr.zr_graph_info(gr)[0] == 1
    zr.zr_graph_launch(gr, stream)
    stream.synchronize()
    assert bool((s.view(torch.uint8) == 0).all())


def test_one_tensor_twice():
    """Inputs may be one tensor: x as its own residual, a matrix times its own transpose, the
    stream's gradient that is also the norm's."""
    device()
    x, _, w, _, _ = layer(130, 128, 516, 5)
    outs = []
    for twin in (x, x.clone()):
        y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(130, device="cuda")
        q, s = zr.fp8_matrix(130, 516)
        zr.zr_rmsnorm_fp8(x, w, y, residual=twin, h=h, rstd=rstd)
        zr.zr_quantize_fp8(y, q, s)
        q2, s2 = (q, s) if twin is x else (q.clone(), s.clone())
        gram = torch.empty(130, 130, device="cuda")
        zr.zr_matmul_fp8(q, s, q2, s2, gram)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        zr.zr_rmsnorm_backward(y, h, w, rstd, dx, dw, zr.rmsnorm_workspace(516), dh=y if twin is x else y.clone())
        outs.append([y, h, rstd, gram, dx, dw])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][3], outs[0][3].t())


def test_views_of_one_buffer():
    """Operands and results that are pieces of one allocation, at odd addresses, side by side."""
    device()
    raw = torch.full((3 * 70 * 301 + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    pieces = [raw[1 + i * 70 * 301:1 + (i + 1) * 70 * 301].view(70, 301) for i in range(3)]
    x, res, w, _, _ = layer(70, 128, 301, 6)
    pieces[0].copy_(x)
    pieces[1].copy_(res)
    y = torch.empty_like(x)
    zr.zr_rmsnorm_fp8(x, w, y, residual=res)
    zr.zr_rmsnorm_fp8(pieces[0], w, pieces[2], residual=pieces[1])
    assert torch.equal(pieces[2], y) and torch.equal(pieces[0], x) and torch.equal(pieces[1], res)
    assert bool(raw[0].isnan()) and bool(raw[1 + 3 * 70 * 301:].isnan().all())
