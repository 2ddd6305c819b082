"""Positions that all axes share (a distance of 0 between them), forward and backward."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from gpu_util import device

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(t, h, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(t, h, d, generator=g, device="cuda").to(BF)


def both(q, k, w, positions, rope, q_out=None, k_out=None):
    """Outputs of the forward pass and the gradients of the outputs themselves."""
    d = q.shape[2]
    q_out, k_out = (torch.empty_like(x, memory_format=torch.contiguous_format) if o is None else o
                    for x, o in ((q, q_out), (k, k_out)))
    x = q.clone(), k.clone()
    zr.zr_qk_norm_rope(q, k, w, w, positions, rope, q_out, k_out)
    out = [q_out.clone(), k_out.clone()]
    dw = [torch.empty(d, dtype=BF, device="cuda") for _ in "qk"]
    dx = [torch.empty_like(x) for x in out]
    zr.zr_qk_norm_rope_backward(*out, *x, w, w, positions, rope, *dx, *dw, zr.qk_norm_workspace(d))
    return out + dx + dw


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t", [1, 2, 37, 3000])
def test_positions_that_all_axes_share(t, interleaved):
    """Text has one position on all axes: an expanded view gives what its copy gives, and what one
    axis gives."""
    device()
    d, freq = 64, 1e4 ** (-torch.arange(0, 64, 2, device="cuda") / 64)
    axis = [j % 3 for j in range(d // 2)]
    q, k, w = rows(t, 6, d, 1), rows(t, 2, d, 2), rows(1, 1, d, 3).view(d)
    one = torch.arange(5, 5 + t, device="cuda")
    rope = zr.rope(freq, interleaved=interleaved, pair_axis=axis)
    shared = one[None].expand(3, t)
    assert shared.stride(0) == 0
    got = both(q, k, w, shared, rope)
    assert all(torch.equal(a, b) for a, b in zip(got, both(q, k, w, shared.contiguous(), rope)))
    assert all(torch.equal(a, b) for a, b in zip(got, both(q, k, w, one, zr.rope(freq, interleaved=interleaved))))
