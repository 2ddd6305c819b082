"""zr_graph_set_adamw with another grad_scale: the captured gradient norm that bounds the step
follows it, so that a replay gives the bits of the eager calls with that scale."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from gpu_util import device

pytestmark = pytest.mark.gpu
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
HP = dict(lr=5e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
SCALES = [0.5, 1.0, 0.125, 3.0]


class Step:
    """norm -> clipped AdamW of one shard, in one list or in two calls (the rank's slice, then
    tensors that every rank holds); `grad_scale` is the norm's and the step's."""

    def __init__(self, dtype, n, apart):
        g = torch.Generator(device="cuda").manual_seed(n)
        self.grad = (torch.randn(n, generator=g, device="cuda") * 1e-3 * (64 if dtype == FP16 else 1)).to(dtype)
        self.st = [torch.randn(n, generator=g, device="cuda") * 0.02, torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
        self.param = torch.empty(n, dtype=dtype, device="cuda")
        self.rec, self.ws, self.ls = zr.clip_record(), zr.grad_norm_workspace(), zr.loss_scale_record()
        zr.zr_loss_scale_init(self.ls, 64.0)
        self.lists = [zr.tensor_list([self.grad[:n // 3]]), zr.tensor_list([self.grad[n // 3:]])] if apart else \
            [zr.tensor_list([self.grad])]

    def run(self, step, grad_scale, norm_scale=None):
        f16 = self.grad.dtype == FP16
        for i, part in enumerate(self.lists):
            zr.zr_grad_norm(part, self.rec, self.ws, max_norm=0.01, grad_scale=grad_scale if norm_scale is None else norm_scale,
                            accumulate=i > 0, ls=self.ls if f16 else None)
        args = (self.grad, *self.st, self.param)
        if f16:
            zr.zr_adamw_step_clip_f16(*args, self.ls, self.rec, step=step, grad_scale=grad_scale, **HP)
        else:
            zr.zr_adamw_step_clip(*args, self.rec, step=step, grad_scale=grad_scale, **HP)

    def outputs(self):
        return [*self.st, self.param.view(torch.int16), self.rec.view(torch.int64)]


def captured(run):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        zr.zr_graph_capture_begin()
        run()
        return zr.zr_graph_capture_end(), side


def replay(graph, side, **hp):
    torch.cuda.synchronize()
    zr.zr_graph_set_adamw(graph, **hp, **HP)
    zr.zr_graph_launch(graph, side)
    side.synchronize()


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("n", [3001, 700_001])  # the norm in one workgroup, and in many
@pytest.mark.parametrize("dtype", [BF, FP16])
def test_norm_follows_the_steps_grad_scale(dtype, n, apart):
    device()
    eager, rec = Step(dtype, n, apart), Step(dtype, n, apart)
    graph, side = captured(lambda: rec.run(1, 1.0))
    assert zr.zr_graph_info(graph)[1] == 1
    factors = set()
    for t, scale in enumerate(SCALES, 1):
        eager.run(t, scale)
        replay(graph, side, step=t, grad_scale=scale)
        for x, y in zip(eager.outputs(), rec.outputs()):
            assert torch.equal(x, y), (t, scale)
        factors.add(rec.rec.view(F32)[3].item())
        torch.ones(1 << 16, device="cuda").sum().item()
    assert len(factors) > 2  # the bound acted, each scale in its own way


def test_norm_of_fp32_beside_the_step():
    """fp32 tensors' norm (their kernel is another), clipped in place, then a step that reads no record."""
    device()
    n = 2000
    x = torch.linspace(-1, 1, n, device="cuda")
    e, r = Step(BF, n, False), Step(BF, n, False)

    def run(s, y, step, scale):
        zr.zr_grad_norm([y], s.rec, s.ws, max_norm=0.5, grad_scale=scale)
        zr.zr_clip_grads([y], s.rec)
        zr.zr_adamw_step(s.grad, *s.st, s.param, step=step, grad_scale=scale, **HP)

    ye, yr = x.clone(), x.clone()
    graph, side = captured(lambda: run(r, yr, 1, 1.0))
    for t, scale in enumerate(SCALES, 1):
        run(e, ye, t, scale)
        replay(graph, side, step=t, grad_scale=scale)
        assert torch.equal(ye, yr)
        assert all(torch.equal(a, b) for a, b in zip(e.outputs(), r.outputs())), (t, scale)


def test_norm_of_another_scale_stays_as_captured():
    """A norm that was captured with a scale that no step of the graph has is not the step's."""
    device()
    eager, rec = Step(BF, 3001, False), Step(BF, 3001, False)
    graph, side = captured(lambda: rec.run(1, 0.5, norm_scale=2.0))
    for t, scale in enumerate(SCALES, 1):
        eager.run(t, scale, norm_scale=2.0)
        replay(graph, side, step=t, grad_scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(eager.outputs(), rec.outputs())), (t, scale)
