"""The accesses of the 8-bit operators that may start at any element say so to the
compiler: no vector is read or written through a type of a larger alignment than its
buffer's (CPU only; the device code is compiled, not run)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "zero_sharded_optimizer_zr_amd"))
import build as zr_build  # noqa: E402

CSRC = os.path.join(ROOT, "zero_sharded_optimizer_zr_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


@pytest.mark.parametrize("src", ["quant_fp8.hip", "rmsnorm.hip", "matmul_fp8.hip"])
def test_no_access_claims_more_alignment_than_its_buffer(src):
    r = subprocess.run(["hipcc", *zr_build.FLAGS, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-fsyntax-only",
                        "--offload-device-only", "-Werror=align-mismatch", os.path.join(CSRC, src)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[:2000]
