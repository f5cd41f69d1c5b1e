"""The convolution reads no input at or behind a row's length, and computes the same with such memory
out of reach: tests/host/conv_reads.cpp, the kernels of csrc/conv_kernels.hip built for the CPU
(tests/host/emulate), with the pages of x behind each row's length closed."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "selective_state_space_fwd_amd", "csrc")
CLANG = shutil.which("clang++") or shutil.which("/opt/rocm/llvm/bin/clang++")


@pytest.mark.skipif(CLANG is None, reason="clang++ not available")
def test_conv_reads(tmp_path):
    # Copies, so that their includes find the CPU's device_math.h and device_scan.h; the empty
    # asm statements pin vector registers and have no meaning here.
    for name, copy in (("conv_kernels.hip", "conv_kernels.cpp"), ("device_block.h", "device_block.h")):
        text = open(os.path.join(CSRC, name)).read()
        (tmp_path / copy).write_text(re.sub(r'asm volatile\(""[^;]*;', ";", text))
    exe = str(tmp_path / "conv_reads")
    cmd = [CLANG, "-std=c++20", "-O1", "-pthread", "-I", os.path.join(HERE, "host", "emulate"), "-I",
           os.path.join(ROOT, "include"), "-I", CSRC, "-o", exe, os.path.join(HERE, "host", "conv_reads.cpp"),
           str(tmp_path / "conv_kernels.cpp"), os.path.join(CSRC, "conv_api.cpp")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    print(r.stdout[-2000:])
    assert r.returncode == 0 and "conv reads ok" in r.stdout, f"{r.returncode}\n{r.stdout[-3000:]}"
