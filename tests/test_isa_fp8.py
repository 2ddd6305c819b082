"""The gfx950 code of the 8-bit operators has the shape their design states (CPU only:
hipcc cross-compiles the device code to assembly here): no kernel spills, products with
16-bit outputs use the scaled 8-bit matrix instructions and the ones with fp32 outputs the
bf16 ones, the LDS kernels load without passing through registers."""
import os
import re
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "zero_sharded_optimizer_zr_amd"))
import build as zr_build  # noqa: E402

CSRC = os.path.join(ROOT, "zero_sharded_optimizer_zr_amd", "csrc")
SOURCES = ["quant_fp8.hip", "rmsnorm.hip", "matmul_fp8.hip"]


@pytest.fixture(scope="module")
def asm():
    tmp = tempfile.mkdtemp(prefix="zr_isa_fp8_")

    def compile_one(name):
        out = os.path.join(tmp, name + ".s")
        cmd = ["hipcc", *zr_build.FLAGS, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
               "--offload-device-only", "-S", os.path.join(CSRC, name), "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        with open(out) as f:
            return name, f.read()

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(pool.map(compile_one, SOURCES))


def body(text, fragment):
    m = re.search(r"^_Z\S*" + re.escape(fragment) + r"\S*:", text, re.M)
    assert m, f"kernel {fragment} not found"
    return text[m.end():text.index(".Lfunc_end", m.end())]


@pytest.mark.parametrize("src", SOURCES)
def test_nothing_spills(asm, src):
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", asm[src])
    assert sizes and set(sizes) == {"0"}
    assert not re.search(r"v_pk_(add|mul|fma)_f32", asm[src])


@pytest.mark.parametrize("kernel,count,instruction", [
    ("matmul_big_kernelILi0E", 32, "v_mfma_scale_f32_32x32x64_f8f6f4"),
    ("matmul_mid_kernelILi0ELb0E", 32, "v_mfma_scale_f32_16x16x128_f8f6f4"),
    ("matmul_mid_kernelILi1ELb1E", 128, "v_mfma_f32_16x16x32_bf16"),
    ("matmul_pair_kernelILi1ELb0E", 16, "v_mfma_scale_f32_16x16x128_f8f6f4"),
    ("matmul_pair_kernelILi0ELb1E", 64, "v_mfma_f32_16x16x32_bf16"),
])
def test_products(asm, kernel, count, instruction):
    """The products of one group (two for the kernels that alternate two sets of registers),
    and loads into LDS."""
    text = body(asm["matmul_fp8.hip"], kernel)
    assert len(re.findall(r"v_mfma\w*", text)) == len(re.findall(re.escape(instruction), text)) == count
    assert re.search(r"buffer_load_dwordx4 .*\blds\b", text)
