"""The grids of all launches (host code): below HIP's 2^32 work items in a dimension, built
host-only and run (tests/host_launch_grid.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_optimizer_zr_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


def test_launch_grids(tmp_path, monkeypatch):
    monkeypatch.delenv("ZR_MAX_GRID", raising=False)
    exe = str(tmp_path / "launch_grid")
    r = subprocess.run(["hipcc", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                        f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(ROOT, "tests", "host_launch_grid.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok:"), (r.stdout + r.stderr)[-2000:]
