"""The head norms and the clipped step together with the calls around them, as a training step
makes them: norm, fused query/key/value product, head norms with rotation, their backward
pass into the product's gradient, weight gradients into flat contributions, mean, global norm over
the slice and the tensors that stay whole, clipped AdamW."""
import threading

import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from fp8_util import E5M2, HALF
from gpu_util import device

pytestmark = pytest.mark.gpu
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
T, HIDDEN, HQ, HK, D = 200, 256, 4, 2, 64
WIDTH = (HQ + 2 * HK) * D


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


class Step:
    """One rank of two, which holds the first half of the flat gradient of W [WIDTH, HIDDEN] and
    all of the two head weights."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        new = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
        self.x, self.w = r(T, HIDDEN).to(BF), (0.08 * r(WIDTH, HIDDEN)).to(BF)
        self.wn, self.wq, self.wk = ((1 + 0.1 * r(n)).to(BF) for n in (HIDDEN, D, D))
        self.dy = (r(T, WIDTH) * 0.1).to(BF)  # of queries, keys (turned) and values
        self.pos = torch.arange(T, device="cuda") % 77 + 1000
        self.rope = zr.rope(1e4 ** (-torch.arange(0, D, 2, device="cuda").float() / D))
        self.norm, self.q8 = new(T, HIDDEN), zr.fp8_matrix(T, HIDDEN)
        self.w8, self.wt8 = zr.fp8_matrix(WIDTH, HIDDEN, block_rows=128), zr.fp8_matrix(HIDDEN, WIDTH, block_rows=128)
        self.qkv, self.dqkv = new(T, WIDTH), new(T, WIDTH)
        self.q_out, self.k_out = new(T, HQ, D), new(T, HK, D)
        self.d8t, self.n8t = zr.fp8_matrix(WIDTH, T, E5M2), zr.fp8_matrix(HIDDEN, T)
        self.ws, self.norm_ws, self.rec = zr.qk_norm_workspace(D), zr.grad_norm_workspace(), zr.clip_record()
        # this rank's contribution, flat: W's gradient; the head weights' gradients behind one another
        n = WIDTH * HIDDEN
        self.flat, self.small = new(n), new(2 * D)
        self.peer, self.peer_small = (r(n) * 0.01).to(BF), (r(2 * D) * 0.01).to(BF)
        self.mean, self.mean_small = new(n // 2), new(2 * D)
        self.list, self.small_list = zr.tensor_list([self.mean]), zr.tensor_list([self.mean_small[:D], self.mean_small[D:]])
        state = lambda m: [0.02 * r(m), torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda")]  # noqa: E731
        self.st, self.st_small, self.param = state(n // 2), state(2 * D), new(n // 2)
        # the other rank's sum of squares, as an all-reduce would bring it
        self.other = torch.tensor([0.75], dtype=torch.float64, device="cuda")

    def heads(self, rows):
        return rows[:, :HQ * D].view(T, HQ, D), rows[:, HQ * D:(HQ + HK) * D].view(T, HK, D)

    def run(self, t, stream=None):
        kw = dict(stream=stream)
        zr.zr_quantize_fp8(self.w, *self.w8, *self.wt8, block_rows=128, **kw)
        zr.zr_rmsnorm_fp8(self.x, self.wn, self.norm, *self.q8, **kw)
        zr.zr_matmul_fp8(*self.q8, *self.w8, self.qkv, b_block_rows=128, **kw)
        zr.zr_qk_norm_rope(*self.heads(self.qkv), self.wq, self.wk, self.pos, self.rope, self.q_out, self.k_out, **kw)
        self.dqkv[:, (HQ + HK) * D:].copy_(self.dy[:, (HQ + HK) * D:])
        zr.zr_qk_norm_rope_backward(*self.heads(self.dy), *self.heads(self.qkv), self.wq, self.wk, self.pos, self.rope,
                                    *self.heads(self.dqkv), self.small[:D], self.small[D:], self.ws, **kw)
        zr.zr_quantize_fp8(self.dqkv, qt=self.d8t[0], scales_t=self.d8t[1], **kw)
        zr.zr_quantize_fp8(self.norm, qt=self.n8t[0], scales_t=self.n8t[1], **kw)
        zr.zr_matmul_fp8(*self.d8t, *self.n8t, self.flat.view(WIDTH, HIDDEN), **kw)
        half = self.mean.numel()
        zr.zr_reduce_slice([self.flat[:half], self.peer[:half]], self.mean, **kw)
        zr.zr_reduce_slice([self.small, self.peer_small], self.mean_small, **kw)
        zr.zr_grad_norm(self.list, self.rec, self.norm_ws, **kw)
        self.rec[:1].add_(self.other)
        zr.zr_grad_norm(self.small_list, self.rec, self.norm_ws, max_norm=0.25, accumulate=True, **kw)
        zr.zr_adamw_step_clip(self.mean, *self.st, self.param, self.rec, step=t, **HP, **kw)
        zr.zr_adamw_step_clip(self.mean_small, *self.st_small, None, self.rec, step=t, **HP, **kw)

    def outputs(self):
        return [x.clone() for x in (self.q_out, self.k_out, self.dqkv, self.small, self.flat, *self.st, *self.st_small, self.param,
                                    self.rec.view(torch.int64))]


def test_gradients_norm_and_step():
    """Gradients against autograd in 64 bits of the same layer from the product's rows on (codes
    are the products' own matter); distances bounded by the outputs' rounding to bf16, twice
    where the product's operands were rounded to codes besides."""
    device()
    s = Step(1)
    before = [x.clone() for x in s.st]
    s.run(1)
    qkv, wq, wk = (x.double().requires_grad_() for x in (s.qkv, s.wq, s.wk))
    half = D // 2
    angle = (s.pos.double()[:, None] * s.rope.inv_freq.double())[:, None]
    c, sn = torch.cos(angle), torch.sin(angle)
    loss = 0.0
    for x, w, dy, out in zip(s.heads(qkv), (wq, wk), s.heads(s.dy), (s.q_out, s.k_out)):
        y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + 1e-5) * w
        a, b = y[..., :half], y[..., half:]
        y = torch.cat((a * c - b * sn, b * c + a * sn), -1)
        assert rel(out, y.detach()) < 1.05 * HALF[BF]
        loss = loss + (y * dy.double()).sum()
    loss = loss + (qkv[:, (HQ + HK) * D:] * s.dy[:, (HQ + HK) * D:].double()).sum()
    loss.backward()
    assert rel(s.dqkv, qkv.grad) < 1.05 * HALF[BF]
    assert rel(s.small, torch.cat((wq.grad, wk.grad))) < 1.05 * HALF[BF]
    want = s.dqkv.double().t() @ s.norm.double()
    assert rel(s.flat.view(WIDTH, HIDDEN), want) < (2.0 ** -4 + 2.0 ** -3) / 3 ** 0.5
    # the norm of everything: the slice, the other rank's share, the tensors that stay whole
    total = float(s.mean.double().square().sum()) + 0.75 + float(s.mean_small.double().square().sum())
    assert s.rec[0].item() == pytest.approx(total, rel=1e-12)
    factor = s.rec.view(F32)[3].item()
    assert factor == pytest.approx(0.25 / (total ** 0.5 + 1e-6), rel=2.0 ** -23) and factor < 1
    param = torch.empty_like(s.param)
    zr.zr_adamw_step(s.mean, *before, param, step=1, grad_scale=factor, **HP)
    assert all(torch.equal(a, b) for a, b in zip([*before, param], [*s.st, s.param]))


def test_captured_step_replays():
    """The whole step as one graph, replayed between eager runs on other data and beside a second
    graph with buffers of its own: every replay is the eager result."""
    device()
    eager, rec, other = Step(2), Step(2), Step(3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for s in (rec, other):
        with torch.cuda.stream(side):
            zr.zr_graph_capture_begin()
            s.run(1)
            graphs.append(zr.zr_graph_capture_end())
    assert zr.zr_graph_info(graphs[0])[1] == 2
    noise = torch.ones(1 << 20, device="cuda")
    for t in range(1, 6):
        for s in (eager, rec):
            s.x.add_(0.125 * t)
            s.pos.add_(t)
        eager.run(t)
        noise.add_(1).sum().item()
        torch.cuda.synchronize()
        zr.zr_graph_set_adamw(graphs[0], step=t, **HP)
        zr.zr_graph_launch(graphs[0], side)
        zr.zr_graph_launch(graphs[1], side)
        side.synchronize()
        for a, b in zip(eager.outputs(), rec.outputs()):
            assert torch.equal(a, b), t


def test_captured_f16_step_with_an_overflow():
    """fp16 gradients, loss scale and clipping in one graph: an infinity in the third step's
    gradient skips it, eagerly and replayed."""
    device()
    n = 50_003

    def make():
        g = torch.Generator(device="cuda").manual_seed(5)
        st = [torch.randn(n, generator=g, device="cuda") * 0.02, torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
        ls = zr.loss_scale_record()
        zr.zr_loss_scale_init(ls, 1024.0)
        return dict(grad=torch.randn(n, generator=g, device="cuda").to(FP16), st=st, ls=ls, rec=zr.clip_record(),
                    ws=zr.grad_norm_workspace(), param=torch.zeros(n, dtype=FP16, device="cuda"))

    def run(b, t):
        zr.zr_grad_norm([b["grad"]], b["rec"], b["ws"], max_norm=0.05, ls=b["ls"])
        zr.zr_adamw_step_clip_f16(b["grad"], *b["st"], b["param"], b["ls"], b["rec"], step=t, **HP)
        zr.zr_loss_scale_update(b["ls"])

    eager, rec = make(), make()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        zr.zr_graph_capture_begin()
        run(rec, 1)
        graph = zr.zr_graph_capture_end()
    assert zr.zr_graph_info(graph)[1] == 1
    x = torch.ones(1 << 20, device="cuda")
    for t in range(1, 6):
        for b in (eager, rec):
            b["grad"].mul_(0.75)
            if t == 3:
                b["grad"][1234] = float("inf")
            elif t == 4:
                b["grad"][1234] = 0.5
        run(eager, t)
        torch.cuda.synchronize()
        zr.zr_graph_set_adamw(graph, step=t, **HP)
        zr.zr_graph_launch(graph, side)
        side.synchronize()
        x.add_(1).sum().item()
        for a, b in zip((*eager["st"], eager["param"], eager["ls"]), (*rec["st"], rec["param"], rec["ls"])):
            assert torch.equal(a, b), t
        assert rec["ls"].tolist()[3] == (1 if t >= 3 else 0)


def test_threads_on_streams_of_their_own():
    device()
    want = []
    for seed in (7, 8, 9):
        s = Step(seed)
        s.run(1)
        want.append(s.outputs())
    steps = [Step(seed) for seed in (7, 8, 9)]
    torch.cuda.synchronize()
    errors = []

    def work(s):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                s.run(1, stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w))
