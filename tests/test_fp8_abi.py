"""CPU tests of the 8-bit operators' entry points (zr_fp8.h): every declared symbol
is exported and bound, every refusal comes back with its documented code before
anything is launched, and calls without work succeed without a GPU."""
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
    text = open(os.path.join(ROOT, "include", "zr_fp8.h")).read()
    names = re.findall(r"^ZR_API\s+[\w\s\*]+?\b(zr_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(zr.FP8_SYMBOLS) and len(names) == 4
    lib = ctypes.CDLL(zr.LIBRARY)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(zr, name)) and name in zr.__all__
    assert f"#define ZR_FP8_GROUP {zr.ZR_FP8_GROUP}\n" in text
    assert f"#define ZR_RMSNORM_PARTIALS {zr.ZR_RMSNORM_PARTIALS}\n" in text


@pytest.mark.parametrize("compiler,std", [("gcc", "c99"), ("g++", "c++11")])
def test_header_is_plain_c(tmp_path, compiler, std):
    src = tmp_path / ("t.c" if compiler == "gcc" else "t.cpp")
    src.write_text('#include "zr_fp8.h"\nint main(void) { return zr_rmsnorm_fp8 && zr_matmul_fp8 ? ZR_BF16 : ZR_E5M2; }\n')
    subprocess.run([compiler, f"-std={std}", "-Wall", "-Wextra", "-pedantic", "-c",
                    f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(tmp_path / "t.o")], check=True)


def call(fn, base, **change):
    args = dict(base)
    for k in change:
        assert k in args, k
    args.update(change)
    return getattr(L, fn)(*args.values())


QUANT = dict(src=at(0), dtype=0, rows=64, cols=256, ld=256, block_rows=1, format=0, q=at(1), ldq=256, scales=at(2),
             qt=at(3), ldqt=64, scales_t=at(4), stream=None)
MATMUL = dict(a=at(0), lda=256, a_scales=at(1), a_format=0, b=at(2), ldb=256, b_scales=at(3), b_block_rows=1, m=64, n=32,
              k=256, out=at(4), out_dtype=0, ldo=32, accumulate=0, stream=None)
NORM = dict(x=at(0), ldx=256, residual=at(1), ldr=256, weight=at(2), dtype=0, rows=64, cols=256, eps=1e-5, h=at(3), ldh=256,
            y=at(4), ldy=256, q=at(5), ldq=256, scales=at(6), rstd=at(7), stream=None)
GRAD = dict(dy=at(0), lddy=256, h=at(1), ldh=256, weight=at(2), rstd=at(3), dh=at(4), lddh=256, dtype=0, rows=64, cols=256,
            dx=at(5), lddx=256, dweight=at(6), workspace=at(7), stream=None)
BIG = 1 << 62


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(format=2), 1), (dict(block_rows=2), 1), (dict(block_rows=0), 1),
    (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(src=None), 1), (dict(q=None), 1), (dict(scales=None), 1),
    (dict(qt=None), 1), (dict(scales_t=None), 1), (dict(q=None, scales=None, qt=None, scales_t=None), 1),
    (dict(ld=255), 1), (dict(ldq=255), 1), (dict(ldqt=63), 1), (dict(ld=BIG), 1), (dict(ldqt=BIG), 1),
    (dict(src=at(0, 1)), 3), (dict(q=at(0, 4)), 1), (dict(scales=at(1, 16383)), 1), (dict(qt=at(1)), 1),
    (dict(scales_t=at(0, 2 * 64 * 256 - 1)), 1), (dict(scales_t=at(2)), 1)])
def test_quantize_refusals(change, code):
    assert call("zr_quantize_fp8", QUANT, **change) == code
    assert "zr_quantize_fp8" in zr.zr_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(a_format=2), 1), (dict(out_dtype=3), 1), (dict(b_block_rows=64), 1), (dict(accumulate=2), 1), (dict(m=-1), 1),
    (dict(n=-1), 1), (dict(k=-1), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(a_scales=None), 1), (dict(b_scales=None), 1),
    (dict(out=None), 1), (dict(lda=255), 1), (dict(ldb=255), 1), (dict(ldo=31), 1), (dict(lda=BIG), 1), (dict(ldo=BIG), 1),
    (dict(out=at(4, 1)), 3), (dict(out=at(4, 2), out_dtype=2), 3), (dict(out=at(0, 256)), 1), (dict(out=at(2, 32 * 256 - 2)), 1),
    (dict(out=at(1)), 1), (dict(out=at(3, 62)), 1)])
def test_matmul_refusals(change, code):
    assert call("zr_matmul_fp8", MATMUL, **change) == code
    assert "zr_matmul_fp8" in zr.zr_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(eps=1e300), 1), (dict(x=None), 1), (dict(weight=None), 1), (dict(q=None), 1),
    (dict(scales=None), 1), (dict(y=None, q=None, scales=None), 1), (dict(residual=None), 1), (dict(ldx=255), 1),
    (dict(ldr=255), 1), (dict(ldh=255), 1), (dict(ldy=255), 1), (dict(ldq=255), 1), (dict(ldx=BIG), 1),
    (dict(x=at(0, 1)), 3), (dict(weight=at(2, 1)), 3), (dict(y=at(4, 1)), 3), (dict(rstd=at(7, 2)), 3),
    (dict(h=at(0), ldx=264), 1), (dict(h=at(1, 2)), 1), (dict(y=at(0)), 1), (dict(y=at(3)), 1), (dict(q=at(4)), 1),
    (dict(scales=at(5)), 1), (dict(rstd=at(2)), 1), (dict(rstd=at(6)), 1)])
def test_norm_refusals(change, code):
    assert call("zr_rmsnorm_fp8", NORM, **change) == code
    assert "zr_rmsnorm_fp8" in zr.zr_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dy=None), 1), (dict(h=None), 1), (dict(weight=None), 1),
    (dict(rstd=None), 1), (dict(dx=None), 1), (dict(dweight=None), 1), (dict(workspace=None), 1), (dict(lddy=255), 1),
    (dict(ldh=255), 1), (dict(lddh=255), 1), (dict(lddx=255), 1), (dict(lddx=BIG), 1), (dict(cols=BIG, lddy=BIG, ldh=BIG, lddh=BIG, lddx=BIG), 1),
    (dict(dy=at(0, 1)), 3), (dict(dweight=at(6, 1)), 3), (dict(workspace=at(7, 2)), 3), (dict(rstd=at(3, 2)), 3),
    (dict(dx=at(0), lddx=264), 1), (dict(dx=at(1)), 1), (dict(dx=at(4, 2)), 1), (dict(dweight=at(2)), 1),
    (dict(workspace=at(5)), 1), (dict(dweight=at(7, 512 * 256 * 4 - 2)), 1)])
def test_norm_backward_refusals(change, code):
    assert call("zr_rmsnorm_backward", GRAD, **change) == code
    assert "zr_rmsnorm_backward" in zr.zr_last_error()


def test_calls_without_work():
    assert call("zr_quantize_fp8", QUANT, rows=0) == 0 and call("zr_quantize_fp8", QUANT, cols=0, src=None) == 0
    assert call("zr_matmul_fp8", MATMUL, m=0) == 0 and call("zr_matmul_fp8", MATMUL, n=0, b=None) == 0
    assert call("zr_matmul_fp8", MATMUL, k=0, accumulate=1) == 0
    assert call("zr_rmsnorm_fp8", NORM, rows=0, x=None) == 0


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def test_binding_refuses_wrong_tensors():
    x, q, s = cpu(4, 256), cpu(4, 256, dtype=E4M3), cpu(4, 2, dtype=E8M0)
    with pytest.raises(ValueError, match="cuda"):
        zr.zr_quantize_fp8(x, q, s)
    for bad, error in (((x.float(), q, s), TypeError), ((x, q.view(torch.uint8), s), TypeError), ((x, q, s.float()), TypeError),
                       ((x, q[:3], s), ValueError), ((x, q, s[:3]), ValueError), ((x.t(), q, s), ValueError),
                       ((x, None, None), ValueError), ((x.view(2, 2, 256), q, s), ValueError), (([1], q, s), TypeError),
                       ((x, q, s, cpu(256, 4, dtype=torch.float8_e5m2), cpu(256, 1, dtype=E8M0)), TypeError),
                       ((x, q, s, cpu(4, 256, dtype=E4M3), cpu(256, 1, dtype=E8M0)), ValueError),
                       ((x, q, s, cpu(256, 4, dtype=E4M3), cpu(255, 1, dtype=E8M0)), ValueError)):
        with pytest.raises(error):
            zr.zr_quantize_fp8(*bad)
    b, sb, out = cpu(8, 256, dtype=E4M3), cpu(8, 2, dtype=E8M0), cpu(4, 8)
    with pytest.raises(ValueError, match="cuda"):
        zr.zr_matmul_fp8(q, s, b, sb, out)
    for bad, error in (((q, s, b.view(torch.float8_e5m2), sb, out), TypeError), ((q, s, b[:, :128], sb, out), ValueError),
                       ((q, s, b, sb[:7], out), ValueError), ((q, s[:3], b, sb, out), ValueError),
                       ((q, s, b, sb, out.t()), ValueError), ((q, s, b, sb, out.double()), TypeError),
                       ((q, s, b.t().contiguous().t(), sb, out), ValueError)):
        with pytest.raises(error):
            zr.zr_matmul_fp8(*bad)
    with pytest.raises(ValueError):  # one row of scales for 8 rows of B
        zr.zr_matmul_fp8(q, s, b, sb[:1], out, b_block_rows=1)
    w, rstd = cpu(256), cpu(4, dtype=torch.float32)
    with pytest.raises(ValueError, match="cuda"):
        zr.zr_rmsnorm_fp8(x, w, q=q, scales=s, rstd=rstd)
    for kw, error in ((dict(y=x.half()), TypeError), (dict(y=x[:2]), ValueError), (dict(q=q, scales=s[:1]), ValueError),
                      (dict(y=x, rstd=rstd[:3]), ValueError), (dict(y=x, rstd=rstd.half()), TypeError),
                      (dict(y=x, residual=x[:, :100]), ValueError), (dict(y=x, residual=x.half()), TypeError)):
        with pytest.raises(error):
            zr.zr_rmsnorm_fp8(x, w, **kw)
    with pytest.raises(ValueError):
        zr.zr_rmsnorm_fp8(x, w[:255], y=cpu(4, 256))
    ws = cpu(512, 256, dtype=torch.float32)
    good = dict(dy=x, h=x, weight=w, rstd=rstd, dx=x, dweight=w, workspace=ws)
    with pytest.raises(ValueError, match="cuda"):
        zr.zr_rmsnorm_backward(**good)
    for kw, error in ((dict(dy=x.half()), TypeError), (dict(dx=x[:3]), ValueError), (dict(workspace=ws[:511]), ValueError),
                      (dict(workspace=ws.half()), TypeError), (dict(dweight=w[:9]), ValueError), (dict(rstd=rstd[:3]), ValueError),
                      (dict(dh=x[:, :8]), ValueError)):
        with pytest.raises(error):
            zr.zr_rmsnorm_backward(**{**good, **kw})


def test_buffers_of_the_binding():
    q, s = zr.fp8_matrix(5, 300, device="cpu")
    assert q.shape == (5, 300) and q.stride(0) == 384 and s.shape == (5, 3) and s.dtype == E8M0
    q, s = zr.fp8_matrix(200, 300, torch.float8_e5m2, 128, device="cpu")
    assert q.dtype == torch.float8_e5m2 and s.shape == (2, 3)
    assert zr.rmsnorm_workspace(70, device="cpu").numel() == 512 * 70
