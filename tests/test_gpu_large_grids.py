"""Work of more than 2^32 work items: the grid is held below that and the kernels loop."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from gpu_util import device

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_heads_of_2_to_26_tokens_and_more():
    """One head of two elements: a workgroup takes four tokens, so that 2^26 tokens are 2^24
    workgroups.  The same bits as in pieces that fit a grid each, and the backward pass undoes
    the turn."""
    device()
    t = (1 << 26) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, 1, 2, generator=g, device="cuda", dtype=F32).to(BF)
    positions = torch.randint(0, 1 << 20, (t,), generator=g, device="cuda")
    w = torch.tensor([1.5, -0.5], device="cuda").to(BF)
    rope = zr.rope(torch.tensor([0.37], device="cuda"))
    out, want = torch.full_like(x, 9.0), torch.full_like(x, 7.0)
    zr.zr_qk_norm_rope(x, None, w, None, positions, rope, out, None)
    for b in range(0, t, 1 << 24):
        e = min(t, b + (1 << 24))
        zr.zr_qk_norm_rope(x[b:e], None, w, None, positions[b:e], rope, want[b:e], None)
    assert torch.equal(out, want)
    dx = torch.full_like(x, 9.0)
    zr.zr_qk_norm_rope_backward(out, None, None, None, None, None, positions, rope, dx, None)
    y = x.float()
    y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-5) * w.float()
    # two roundings to bf16 of both elements of the pair, at most half a step (2^-8) each
    assert bool(((dx.float() - y).abs() <= 2.5 * 2.0 ** -8 * y.abs().sum(-1, keepdim=True) + 1e-30).all())


def test_clipped_adamw_of_2_to_32_elements_and_more():
    """States whose 16-byte phases disagree go element by element, a thread to each.  The first
    moment of a zero state is (1 - beta1) * gradient * factor, rounded once; half of it
    with a factor of 0.5."""
    device()
    n = (1 << 32) + 7
    grad = torch.full((n + 1,), 2.0, dtype=BF, device="cuda")[1:]
    master, m, v = torch.zeros(n, device="cuda"), torch.zeros(n + 1, device="cuda")[1:], torch.zeros(n, device="cuda")
    rec = torch.zeros(2, dtype=torch.float64, device="cuda")
    rec.view(F32)[2:] = torch.tensor([1.0, 0.5], device="cuda")
    zr.zr_adamw_step_clip(grad, master, m, v, None, rec, step=1, lr=0.5, beta1=0.75, beta2=0.5, eps=1e-8, weight_decay=0.0)
    for state, value in ((m, 0.25), (v, 0.5)):
        assert state[0].item() == value
        for part in state.split(1 << 29):
            assert bool((part == value).all())
    assert bool((master[-8:] == master[0]).all()) and master[0].item() == pytest.approx(-0.5, rel=1e-6)
