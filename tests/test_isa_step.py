"""The gfx950 code of the clipping and head-norm kernels has the shape their design states
(CPU only: hipcc cross-compiles the device code to assembly here): whole vectors, no
scratch, no packed fp32, the streams past the caches."""
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
SOURCES = ["clip.hip", "head_norm.hip"]


@pytest.fixture(scope="module")
def asm():
    tmp = tempfile.mkdtemp(prefix="zr_isa_step_")

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
    lines = [ln.split(";")[0].strip() for ln in text[m.end():text.index(".Lfunc_end", m.end())].splitlines()]
    return [ln for ln in lines if ln and not ln.startswith(".")]


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_and_no_packed_fp32(asm, src):
    """Single elements, four chunks to a lane, backward: heads past 128 elements of which at most
    six are turned.  Their masks are more than the scalar registers hold."""
    sizes = re.findall(r"\.name:\s+(\S+).*?\.private_segment_fixed_size:\s+(\d+)", asm[src], re.S)
    assert sizes
    for name, size in sizes:
        assert size == "0" or "Li1ELi64ELi4E" in name, name
    assert not re.search(r"v_pk_(add|mul|fma)_f32", asm[src])
    assert not re.search(r"\b(s_store|s_buffer_store|s_atomic|global_atomic|flat_atomic)", asm[src])


@pytest.mark.parametrize("kernel,loads,stores", [
    ("squares_kernelINS_4BF16E", 8, 0), ("squares_kernelINS_3F32E", 8, 0), ("clip_kernelINS_4BF16E", 8, 8),
    ("clip_kernelINS_3F16E", 8, 8), ("adamw_clip_vec_kernelINS_8StepBF16ELb1E", 3, 3)])
def test_streams(asm, kernel, loads, stores):
    """A whole tile's 16-byte accesses (AdamW's three states) carry the non-temporal hint; those
    of a tile's edges come beside them."""
    ops = body(asm["clip.hip"], kernel)
    for op, want in (("global_load_dwordx4", loads), ("global_store_dwordx4", stores)):
        lines = [ln for ln in ops if ln.startswith(op)]
        assert len(lines) >= want and all(ln.rstrip().endswith(" nt") for ln in lines), (op, len(lines))
    assert not [ln for ln in ops if ln.startswith(("flat_load", "flat_store", "scratch_"))]


@pytest.mark.parametrize("kernel,width,loads", [
    ("rope_kernelINS_4BF16ELi4ELi16ELi1ELb0ELi4E", "dwordx2", 8 + 2), ("rope_kernelINS_3F16ELi4ELi16ELi1ELb0ELi4E", "dwordx2", 8 + 2),
    ("rope_grad_kernelINS_4BF16ELi8ELi8ELi1ELb0E", "dwordx4", 2 * 4 + 2)])
def test_head_rows(asm, kernel, width, loads):
    """Two vectors to a lane and step (forward four steps at once; backward of the gradient and
    of the row, the first step's and the next one's), two of the weight; two stores a step."""
    ops = body(asm["head_norm.hip"], kernel)
    assert len([ln for ln in ops if ln.startswith(f"global_load_{width}")]) >= loads
    out = [ln for ln in ops if ln.startswith(f"global_store_{width}")]
    assert out and all(ln.rstrip().endswith(" nt") for ln in out)
    assert not [ln for ln in ops if ln.startswith(("flat_load", "flat_store", "scratch_"))]


@pytest.mark.parametrize("src", SOURCES)
def test_memory_is_written_by_vector_and_lds_instructions_alone(asm, src):
    """Every store and every atomic is a global_ or a ds_ one (scratch_ where a kernel spills, which
    the next test bounds), and nothing acts on the scalar cache but its loads."""
    ops = {ln.split()[0] for ln in asm[src].splitlines() if re.match(r"\s+[a-z]\w+", ln)}
    writes = {op for op in ops if "store" in op or "atomic" in op or "write" in op}
    allowed = ("global_store_", "ds_", "v_writelane_", "scratch_store_")
    assert any(op.startswith("global_store_") for op in writes)
    assert not [op for op in writes if not op.startswith(allowed)]
    assert not [op for op in ops if "dcache" in op]


@pytest.mark.parametrize("src", SOURCES)
def test_scratch_of_the_one_spilling_kernel(asm, src):
    """Only the backward kernel of single elements, four chunks to a lane, has scratch, and 32 bytes at most."""
    sizes = re.findall(r"\.name:\s+(\S+).*?\.private_segment_fixed_size:\s+(\d+)", asm[src], re.S)
    assert sizes
    for name, size in sizes:
        spills = "rope_grad_kernel" in name and "Li1ELi64ELi4E" in name
        assert int(size) <= (32 if spills else 0), (name, size)
