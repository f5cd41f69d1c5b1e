"""The C-ABI argument checks of the operators around the scan under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/sanitize/block_harness.cpp, with the launches
stubbed, on valid problems and on sizes and strides at the edges of int64."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "selective_state_space_fwd_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_block_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "block_harness")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", exe,
           os.path.join(HERE, "sanitize", "block_harness.cpp"),
           *(os.path.join(CSRC, f) for f in ("conv_api.cpp", "step_api.cpp", "norm_api.cpp"))]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"build failed:\n{r.stderr[-3000:]}"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    print(r.stdout[-2000:], r.stderr[-4000:])
    assert r.returncode == 0 and "block harness ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
