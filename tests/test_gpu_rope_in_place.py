"""In-place heads of zr_qk_norm_rope and its backward pass whose strides differ only along axes of
length 1."""
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


@pytest.mark.parametrize("t,hq,hk", [(1, 4, 2), (7, 1, 1), (1, 1, 1)])
def test_in_place_along_axes_of_length_one(t, hq, hk):
    """Where a tensor has one token (or one head), the distance of its tokens (heads) means nothing:
    an output that lies where its input does is in place whatever the distance says."""
    device()
    d = 64
    rope = zr.rope(1e4 ** (-torch.arange(0, d, 2, device="cuda") / d))
    positions, w = torch.arange(t, device="cuda") + 3, rows(1, 1, d, 3).view(d)
    q, k = rows(t, hq, d, 1), rows(t, hk, d, 2)
    want = both(q, k, w, positions, rope)

    def other(x):
        s = list(x.stride())
        for axis in (0, 1):
            if x.shape[axis] == 1:
                s[axis] = 5 * s[axis] + 8
        return x.as_strided(x.shape, s)

    assert other(q).stride() != q.stride()
    got = both(q, k, w, positions, rope, other(q), other(k))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the backward pass over the output's gradient, and over the input
    for place in ("dy", "x"):
        dy, x = rows(t, hq, d, 8), rows(t, hq, d, 9)
        dx, dw = torch.empty_like(x), torch.empty(d, dtype=BF, device="cuda")
        ws = zr.qk_norm_workspace(d)
        zr.zr_qk_norm_rope_backward(dy, None, x, None, w, None, positions, rope, dx, None, dw, None, ws)
        to = other(dy if place == "dy" else x)
        zr.zr_qk_norm_rope_backward(dy, None, x, None, w, None, positions, rope, to, None, dw, None, ws)
        assert torch.equal(to, dx)
