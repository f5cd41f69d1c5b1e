"""The operators around the scan refuse, before any HIP call, what a HIP grid cannot take (2^32
work-items or more along an axis), and nothing else for it: tests/host/launch_limits.cpp over the
C-ABI layer with the launches stubbed."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "selective_state_space_fwd_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_launch_limits(tmp_path):
    exe = str(tmp_path / "launch_limits")
    cmd = ["g++", "-std=c++17", "-O1", "-ftrapv", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", exe,
           os.path.join(HERE, "host", "launch_limits.cpp"),
           *(os.path.join(CSRC, f) for f in ("conv_api.cpp", "step_api.cpp", "norm_api.cpp"))]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "launch limits ok" in r.stdout, r.stdout[-3000:] + r.stderr[-1000:]
