"""Assembly statements of the 8-bit product name every register they write, and nothing else in
its kernels uses the one they share with the compiler, m0 (CPU only: the sources
are compiled to IR and to assembly, not run)."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "zero_sharded_optimizer_zr_amd"))
import build as zr_build  # noqa: E402

CSRC = os.path.join(ROOT, "zero_sharded_optimizer_zr_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


def compiled(tmp_path, *flags):
    out = str(tmp_path / "out")
    r = subprocess.run(["hipcc", *zr_build.FLAGS, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "--offload-device-only",
                        "-S", *flags, os.path.join(CSRC, "matmul_fp8.hip"), "-o", out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        return f.read()


def test_statements_that_set_m0_say_so(tmp_path):
    calls = re.findall(r'asm sideeffect "([^"]*)", "([^"]*)"', compiled(tmp_path, "-emit-llvm"))
    setting = [c for c in calls if re.search(r"\bm0\b", c[0])]
    assert setting and all("~{m0}" in c[1] for c in setting)


def test_nothing_else_uses_m0(tmp_path):
    text = re.sub(r";\s*#?ASMSTART.*?;\s*#?ASMEND", "", compiled(tmp_path), flags=re.S)
    assert not re.search(r"^\s+[a-z].*\bm0\b", text, re.M)
