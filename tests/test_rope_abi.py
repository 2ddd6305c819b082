"""CPU tests of the head norms' entry points (zr_rope.h): every declared symbol is exported
and bound, every refusal comes back with its documented code before anything is launched,
and calls without work succeed without a GPU."""
import ctypes
import os
import re

import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = zr._lib
A = 0x7000_0000_0000  # addresses that no call dereferences on the host
T, HQ, HK, D = 10, 4, 2, 16
ROW = (HQ + 2 * HK) * D  # a fused row: queries, keys, values


def at(i, off=0):
    """The i-th of a row of far-apart buffers."""
    return A + i * (1 << 40) + off


class Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("heads", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


def heads(i, n, off=0, token=None, head=D):
    return Heads(at(i, off), n, n * D if token is None else token, head)


def rope(rot=D, axes=1, axis=None, interleaved=0, inv_freq=at(8)):
    keep = None if axis is None else (ctypes.c_uint8 * max(1, len(axis)))(*axis)
    r = zr._Rope(inv_freq, None if keep is None else ctypes.addressof(keep), rot, axes, interleaved)
    r.keep = keep
    return r


FORWARD = dict(q=heads(0, HQ), k=heads(1, HK), q_weight=at(2), k_weight=at(3), dtype=0, tokens=T, head_dim=D, eps=1e-5,
               positions=at(4), position_stride=T, rope=rope(), q_out=heads(5, HQ), k_out=heads(6, HK), stream=None)
BACKWARD = dict(dq=heads(10, HQ), dk=heads(11, HK), **{k: FORWARD[k] for k in list(FORWARD)[:11]}, dq_in=heads(5, HQ),
                dk_in=heads(6, HK), dq_weight=at(12), dk_weight=at(13), workspace=at(14), stream=None)


def call(fn, base, **change):
    args = dict(base)
    for k in change:
        assert k in args, k
    args.update(change)
    return getattr(L, fn)(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in args.values()])


def test_declared_symbols_are_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "zr_rope.h")).read()
    names = re.findall(r"^ZR_API\s+[\w\s\*]+?\b(zr_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(zr.ROPE_SYMBOLS) and len(names) == 2
    lib = ctypes.CDLL(zr.LIBRARY)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(zr, name)) and name in zr.__all__
    for name in ("ZR_MAX_HEAD_DIM", "ZR_MAX_ROPE_AXES", "ZR_QK_PARTIALS"):
        assert f"#define {name} {getattr(zr, name)}\n" in text


BOTH = [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(tokens=-1), 1), (dict(tokens=(1 << 40) + 1), 1), (dict(head_dim=0), 1), (dict(head_dim=513), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=1e300), 1), (dict(rope=None), 1),
    (dict(rope=rope(rot=-2)), 1), (dict(rope=rope(rot=3)), 1), (dict(rope=rope(rot=D + 2)), 1), (dict(rope=rope(axes=0)), 1),
    (dict(rope=rope(axes=5)), 1), (dict(rope=rope(interleaved=2)), 1), (dict(rope=rope(axis=[0] * 7 + [1])), 1),
    (dict(rope=rope(inv_freq=None)), 1), (dict(rope=rope(inv_freq=at(8, 2))), 3), (dict(positions=None), 1),
    (dict(positions=at(4, 4)), 3), (dict(rope=rope(axes=2), position_stride=T - 1), 1),
    (dict(rope=rope(axes=2), position_stride=1 << 61), 1), (dict(q_weight=at(2, 1)), 3), (dict(k_weight=at(3, 1)), 3),
    (dict(q=None), 1), (dict(k=Heads(None, HK, HK * D, D)), 1), (dict(q=heads(0, HQ, off=1)), 3),
    (dict(q=heads(0, HQ, token=HQ * D - 1)), 1), (dict(q=heads(0, HQ, head=D - 1)), 1), (dict(q=heads(0, HQ, token=-64)), 1),
    (dict(q=heads(0, HQ, token=1 << 62)), 1), (dict(q=heads(0, HQ, head=1 << 62)), 1),
    (dict(q=heads(0, HQ, token=D, head=T * D - 1)), 1), (dict(q=heads(0, HQ, token=0, head=0)), 1)]


@pytest.mark.parametrize("change,code", [c for c in BOTH if c[0] != dict(q=None)] + [
    (dict(q_out=None), 1), (dict(k_out=heads(6, HK + 1)), 1), (dict(q=heads(0, -1)), 1), (dict(q=heads(0, 65537)), 1),
    (dict(q_out=heads(0, HQ, off=2)), 1), (dict(q_out=heads(1, HQ)), 1),                       # over q, shifted; over k
    (dict(q_out=heads(0, HQ, token=2 * HQ * D)), 1),                                           # q's address, another stride
    (dict(k_out=heads(5, HK, off=32)), 1), (dict(q_out=heads(2, HQ)), 1), (dict(k_out=heads(3, HK)), 1),
    (dict(k_out=heads(4, HK, off=T * 8 - 2)), 1), (dict(q_out=heads(8, HQ, off=30)), 1),
    (dict(q=heads(0, HQ, token=ROW), k=heads(0, HK, off=2 * HQ * D, token=ROW),
          q_out=heads(0, HQ, token=ROW), k_out=heads(0, HK, off=2 * HQ * D - 2, token=ROW)), 1),  # one element into q
    (dict(q_out=heads(5, HQ, token=ROW), k_out=heads(5, HK, off=2 * (ROW - HK * D + 1), token=ROW)), 1)])
def test_forward_refusals(change, code):
    assert call("zr_qk_norm_rope", FORWARD, **change) == code
    assert "zr_qk_norm_rope" in zr.zr_last_error()


@pytest.mark.parametrize("change,code", BOTH + [
    (dict(dq=Heads(None, HQ, HQ * D, D)), 1), (dict(dk_in=None), 1), (dict(dq_weight=None), 1), (dict(dk_weight=None), 1),
    (dict(workspace=None), 1), (dict(dq_weight=at(12, 1)), 3), (dict(workspace=at(14, 2)), 3), (dict(q=heads(0, HQ - 1)), 1),
    (dict(dq=heads(10, 65537)), 1), (dict(dk_weight=at(12, 2)), 1), (dict(dq_weight=at(14)), 1), (dict(dq_weight=at(2)), 1),
    (dict(dq_in=heads(14, HQ)), 1), (dict(dq_in=heads(10, HQ, off=2)), 1), (dict(dq_in=heads(1, HQ)), 1),
    (dict(workspace=at(0)), 1), (dict(dk_in=heads(0, HK)), 1), (dict(dk_in=heads(4, HK)), 1)])
def test_backward_refusals(change, code):
    assert call("zr_qk_norm_rope_backward", BACKWARD, **change) == code
    assert "zr_qk_norm_rope_backward" in zr.zr_last_error()


def test_calls_without_work():
    none = Heads(None, 0, 0, 0)
    assert call("zr_qk_norm_rope", FORWARD, tokens=0) == 0
    assert call("zr_qk_norm_rope", FORWARD, tokens=0, q=None, k=None, positions=None, q_out=None, k_out=None) == 0
    assert call("zr_qk_norm_rope", FORWARD, q=None, k=none, q_out=None, k_out=None) == 0
    # no weight, no tokens: nothing to write
    nothing = dict(q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, workspace=None)
    assert call("zr_qk_norm_rope_backward", BACKWARD, tokens=0, **nothing) == 0
    assert call("zr_qk_norm_rope_backward", BACKWARD, dq=None, dk=none, **nothing) == 0


@pytest.mark.parametrize("fn,base", [("zr_qk_norm_rope", FORWARD), ("zr_qk_norm_rope_backward", BACKWARD)])
def test_positions_that_all_axes_share(fn, base):
    """A distance of 0 is no refusal, one between 0 and the tokens is; the shared row counts as a
    buffer (the outputs over its first and its last position)."""
    out = "k_out" if fn == "zr_qk_norm_rope" else "dk_in"
    shared = dict(rope=rope(axes=3, axis=[0, 1, 2, 0, 1, 2, 0, 1]), position_stride=0)
    for stride in (1, T - 1, -1):
        assert call(fn, base, **{**shared, "position_stride": stride}) == 1
        assert "position_stride" in zr.zr_last_error()
    for off in (0, T * 8 - 2):
        assert call(fn, base, **shared, **{out: heads(4, HK, off=off)}) == 1
        assert "overlaps" in zr.zr_last_error()


# ------------------------------------------------------------------- binding ----

def tensors(t=3):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return dict(q=bf(t, 4, 8), k=bf(t, 2, 8), q_weight=bf(8), k_weight=bf(8), positions=torch.arange(t), rope=zr.rope(torch.ones(4)),
                q_out=bf(t, 4, 8), k_out=bf(t, 2, 8))


@pytest.mark.parametrize("change,error", [
    (dict(), ValueError),  # host tensors
    (dict(q=torch.zeros(3, 4, 8)), TypeError), (dict(k=torch.zeros(3, 2, 8, dtype=torch.float16)), TypeError),
    (dict(q=torch.zeros(3, 32, dtype=torch.bfloat16)), ValueError), (dict(k=torch.zeros(2, 2, 8, dtype=torch.bfloat16)), ValueError),
    (dict(q=None, k=None), ValueError), (dict(q_out=torch.zeros(3, 4, 9, dtype=torch.bfloat16)[..., :7]), ValueError),
    (dict(q_weight=torch.zeros(7, dtype=torch.bfloat16)), ValueError), (dict(k_weight=torch.zeros(8)), TypeError),
    (dict(positions=torch.arange(3, dtype=torch.int32)), TypeError), (dict(positions=torch.arange(4)), ValueError),
    (dict(positions=torch.zeros(2, 4, dtype=torch.int64)), ValueError), (dict(positions=[0, 1, 2]), TypeError),
    (dict(rope=zr.rope(torch.ones(4), pair_axis=[0, 0, 1, 1])), ValueError),  # two axes, positions of one
    (dict(q=torch.zeros(3, 4, 16, dtype=torch.bfloat16)[..., ::2]), ValueError)])
def test_binding_refusals(change, error):
    with pytest.raises(error):
        zr.zr_qk_norm_rope(**{**tensors(), **change})


def test_binding_backward_refuses():
    t = tensors()
    args = dict(dq=t["q_out"], dk=t["k_out"], q=t["q"], k=t["k"], q_weight=t["q_weight"], k_weight=t["k_weight"],
                positions=t["positions"], rope=t["rope"], dq_in=t["q"], dk_in=t["k"], dq_weight=t["q_weight"],
                dk_weight=t["k_weight"], workspace=torch.zeros(zr.ZR_QK_PARTIALS, 8))
    for change in (dict(), dict(workspace=torch.zeros(zr.ZR_QK_PARTIALS * 8 - 1)), dict(q=t["q"][:2]), dict(dq=None, dk=None),
                   dict(dq_weight=t["q_weight"][:4])):
        with pytest.raises(ValueError):
            zr.zr_qk_norm_rope_backward(**{**args, **change})


def test_rope_checks():
    with pytest.raises(ValueError):
        zr.rope(torch.ones(257))
    with pytest.raises(ValueError):
        zr.rope(torch.ones(4), pair_axis=[0, 1])
    with pytest.raises(ValueError):
        zr.rope(torch.ones(4), pair_axis=[0, 1, 2, 4])
    with pytest.raises(TypeError):
        zr.rope(torch.ones(4, dtype=torch.float64))
    r = zr.rope(torch.ones(4), interleaved=True, pair_axis=[0, 2, 1, 0])
    assert (r.c.rot_dim, r.c.axes, r.c.interleaved) == (8, 3, 1)
