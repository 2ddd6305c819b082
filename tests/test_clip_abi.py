"""CPU tests of the clipping calls' entry points (zr_clip.h): every declared symbol is
exported and bound, every refusal comes back with its documented code before anything is
launched, and calls without work succeed without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = zr._lib
A = 0x7000_0000_0000  # addresses that no call dereferences on the host


def at(i, off=0):
    """The i-th of a row of far-apart buffers."""
    return A + i * (1 << 40) + off


def test_declared_symbols_are_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "zr_clip.h")).read()
    names = re.findall(r"^ZR_API\s+[\w\s\*]+?\b(zr_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(zr.CLIP_SYMBOLS) and len(names) == 4
    lib = ctypes.CDLL(zr.LIBRARY)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(zr, name)) and name in zr.__all__
    assert f"#define ZR_GRAD_NORM_PARTIALS {zr.ZR_GRAD_NORM_PARTIALS}\n" in text
    assert all(hasattr(zr, name) for name in zr.__all__)


@pytest.mark.parametrize("header,name", [("zr_clip.h", "zr_grad_norm"), ("zr_rope.h", "zr_qk_norm_rope")])
@pytest.mark.parametrize("compiler,std", [("gcc", "c99"), ("g++", "c++11")])
def test_headers_are_plain_c(tmp_path, compiler, std, header, name):
    src = tmp_path / ("t.c" if compiler == "gcc" else "t.cpp")
    src.write_text(f'#include "{header}"\nint main(void) {{ return {name} ? ZR_BF16 : ZR_F32; }}\n')
    subprocess.run([compiler, f"-std={std}", "-Wall", "-Wextra", "-pedantic", "-c",
                    f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(tmp_path / "t.o")], check=True)


def pieces(*items):
    """(pointers, element counts) of (address, count) pairs."""
    return (ctypes.c_void_p * max(1, len(items)))(*[p for p, _ in items]), \
        (ctypes.c_int64 * max(1, len(items)))(*[n for _, n in items])


def norm(items=((at(0), 100), (at(1), 7)), dtype=0, max_norm=1.0, eps=1e-6, grad_scale=1.0, accumulate=0, ls=at(3),
         clip=at(4), workspace=at(5), n=None, hp=True, lists=True):
    ptrs, numels = pieces(*items)
    h = zr._ClipHParams(max_norm, eps, grad_scale)
    return L.zr_grad_norm(ptrs if lists else None, numels if lists else None, len(items) if n is None else n, dtype,
                          ctypes.byref(h) if hp else None, accumulate, ls, clip, workspace, None)


inf, nan = float("inf"), float("nan")
WORK = 8 * zr.ZR_GRAD_NORM_PARTIALS


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(n=-1), 1), (dict(lists=False), 1), (dict(hp=False), 1),
    (dict(max_norm=0.0), 1), (dict(max_norm=-1.0), 1), (dict(max_norm=nan), 1), (dict(eps=-1e-9), 1), (dict(eps=inf), 1),
    (dict(eps=nan), 1), (dict(grad_scale=inf), 1), (dict(grad_scale=nan), 1), (dict(accumulate=2), 1),
    (dict(clip=None), 1), (dict(workspace=None), 1), (dict(clip=at(4, 4)), 3), (dict(workspace=at(5, 4)), 3),
    (dict(ls=at(3, 2)), 3), (dict(items=((at(0), -1),)), 1), (dict(items=((None, 1),)), 1),
    (dict(items=((at(0), (1 << 42) + 1),)), 1), (dict(items=((at(0, 1), 8),)), 3),
    (dict(items=((at(0, 2), 8),), dtype=2), 3), (dict(clip=at(5, WORK - 8)), 1), (dict(ls=at(4, 12)), 1),
    (dict(ls=at(5, WORK - 4)), 1), (dict(items=((at(4, -18), 10),)), 1), (dict(items=((at(5, WORK - 2), 10),)), 1),
    (dict(items=((at(0), 5), (at(3, -2), 2),)), 1)])
def test_norm_refusals(change, code):
    assert norm(**change) == code
    assert "zr_grad_norm" in zr.zr_last_error()


def clip(items=((at(0), 100), (at(1), 7)), dtype=0, record=at(4), n=None):
    ptrs, numels = pieces(*items)
    return L.zr_clip_grads(ptrs, numels, len(items) if n is None else n, dtype, record, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), 1), (dict(n=-1), 1), (dict(record=None), 1), (dict(record=at(4, 4)), 3),
    (dict(items=((at(0), -1),)), 1), (dict(items=((None, 1),)), 1), (dict(items=((at(0, 1), 8),)), 3),
    (dict(items=((at(4, 14), 10),)), 1), (dict(items=((at(0), 8), (at(0), 8))), 1),          # the same tensor twice
    (dict(items=((at(0, 16), 8), (at(2), 8), (at(0), 9))), 1),                               # out of order, one element shared
    (dict(items=((at(0), 8), (at(0, 12), 8))), 1), (dict(items=((at(0), 4), (at(0, 12), 1)), dtype=2), 1)])
def test_clip_refusals(change, code):
    assert clip(**change) == code
    assert "zr_clip_grads" in zr.zr_last_error()


def test_lists_without_work():
    """Nothing to scale: no launch, whatever the order of the empty tensors."""
    assert clip(items=()) == 0
    assert clip(items=((None, 0), (at(0), 0), (at(0), 0))) == 0


HP = zr._HParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, 1)


def adamw(f16=False, grad=at(0), master=at(1), m=at(2), v=at(3), param=at(4), numel=100, hp=HP, ls=at(6), record=at(5)):
    args = (grad, master, m, v, param, numel, None if hp is None else ctypes.byref(hp))
    return L.zr_adamw_step_clip_f16(*args, ls, record, None) if f16 else L.zr_adamw_step_clip(*args, record, None)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(hp=None), 1), (dict(hp=zr._HParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, 0)), 1),
    (dict(hp=zr._HParams(1e-3, 1.0, 0.999, 1e-8, 0.0, 1.0, 1)), 1), (dict(numel=-1), 1), (dict(grad=None), 1),
    (dict(master=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(record=None), 1), (dict(record=at(5, 4)), 3),
    (dict(grad=at(0, 1)), 3), (dict(param=at(4, 1)), 3), (dict(master=at(1, 2)), 3), (dict(master=at(0, 196)), 1),
    (dict(record=at(1, 392)), 1), (dict(record=at(4, 192)), 1), (dict(param=at(0)), 1)])
def test_adamw_refusals(f16, change, code):
    assert adamw(f16, **change) == code
    assert ("zr_adamw_step_clip_f16" if f16 else "zr_adamw_step_clip") in zr.zr_last_error()


@pytest.mark.parametrize("change,code", [(dict(ls=None), 1), (dict(ls=at(6, 2)), 3), (dict(ls=at(5, 8)), 1),
                                         (dict(ls=at(3, 384)), 1)])
def test_adamw_f16_refusals(change, code):
    assert adamw(True, **change) == code


def test_adamw_without_elements():
    assert adamw(numel=0) == 0 and adamw(True, numel=0) == 0
    assert adamw(numel=0, grad=None, master=None, m=None, v=None, param=None) == 0


# ------------------------------------------------------------------- binding ----

def test_binding_refuses_host_tensors():
    bf, f32, rec, ws = torch.zeros(8, dtype=torch.bfloat16), torch.zeros(8), torch.zeros(2, dtype=torch.float64), \
        torch.zeros(zr.ZR_GRAD_NORM_PARTIALS, dtype=torch.float64)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    ls = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: zr.zr_grad_norm([bf], rec, ws), lambda: zr.zr_grad_norm([], rec, ws),
                 lambda: zr.zr_clip_grads([bf], rec), lambda: zr.zr_adamw_step_clip(bf, f32, f32, f32, bf, rec, **hp),
                 lambda: zr.zr_adamw_step_clip_f16(bf, f32, f32, f32, bf, ls, rec, **hp)):
        with pytest.raises(ValueError, match="cuda tensor"):
            call()


def test_binding_checks_lists_and_sizes():
    bf, rec = torch.zeros(8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.float64)
    ws = torch.zeros(zr.ZR_GRAD_NORM_PARTIALS, dtype=torch.float64)
    with pytest.raises(TypeError):
        zr.tensor_list([bf, torch.zeros(8)])                      # two dtypes
    with pytest.raises(TypeError):
        zr.tensor_list([torch.zeros(8, dtype=torch.float64)])
    with pytest.raises(TypeError):
        zr.tensor_list([bf, [1.0]])
    with pytest.raises(ValueError):
        zr.tensor_list([torch.zeros(8, 8, dtype=torch.bfloat16)[:, :4]])
    with pytest.raises(ValueError):
        zr.zr_grad_norm([bf], rec, ws[:-1])
    with pytest.raises(ValueError):
        zr.zr_grad_norm([bf], rec[:1], ws)
    with pytest.raises(TypeError):
        zr.zr_grad_norm([bf], torch.zeros(4), ws)
    with pytest.raises(TypeError):
        zr.zr_grad_norm([bf], rec, ws.float())
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    f32 = torch.zeros(8)
    with pytest.raises(ValueError):
        zr.zr_adamw_step_clip(bf[:7], f32, f32, f32, bf, rec, **hp)
    kept = zr.tensor_list([bf, bf[:3], bf[:0]])
    assert len(kept) == 3 and list(kept.numels) == [8, 3, 0]
