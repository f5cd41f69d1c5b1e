"""The kernels of linear attention and of the queries' and keys' norm built for the CPU
(tests/host/linattn.cpp, tests/host/emulate_mma): values against plain loops in 64 bits, no access
outside any array, nothing read behind a row's length."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "selective_state_space_fwd_amd", "csrc")
CLANG = shutil.which("clang++") or shutil.which("/opt/rocm/llvm/bin/clang++")
KERNELS = ("linattn_kernels.hip", "linattn_bwd.hip", "linattn_step.hip", "qk_kernels.hip")


HOST = ("linattn_api.cpp", "qk_api.cpp")
# Launch rules that send these small cases down the ways of large calls: states left by a walk, segments
# of few chunks, several heads a lane group, workgroups that stay for many items.
LARGE = {"kLinattnCached": 0, "kLinattnWhole": 1, "kQkManyWaves": 1, "kQkMostPartials": 3}


def build(folder, rules={}):
    # Copies, so that their includes find the CPU's device_math.h and device_scan.h.
    found = set()
    for name in (*KERNELS, *HOST, "device_block.h", "device_linattn.h", "linattn_launch.h", "qk_launch.h",
                 "heads.h"):
        text = open(os.path.join(CSRC, name)).read()
        for rule, value in rules.items():
            text, n = re.subn(rf"(constexpr int64_t {rule} =)[^;]*;", rf"\1 {value};", text)
            found |= {rule} if n else set()
        text = re.sub(r'asm volatile\("s_waitcnt[^;]*;', "__syncthreads();", text)
        text = text.replace("__attribute__((address_space(3)))", "")
        with open(os.path.join(folder, name.replace(".hip", ".cpp")), "w") as f:
            f.write(text)
    assert found == set(rules)
    exe = os.path.join(folder, "linattn")
    flags = [CLANG, "-std=c++20", "-O1", "-fno-unroll-loops", "-Wno-everything", "-I",
             os.path.join(HERE, "host", "emulate_mma"), "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    sources = [os.path.join(HERE, "host", "linattn.cpp")]
    sources += [os.path.join(folder, k.replace(".hip", ".cpp")) for k in (*HOST, *KERNELS)]
    objects = [os.path.join(folder, os.path.basename(s) + ".o") for s in sources]
    jobs = [subprocess.Popen([*flags, "-c", s, "-o", o], stderr=subprocess.PIPE, text=True)
            for s, o in zip(sources, objects)]
    for j in jobs:
        _, err = j.communicate()
        assert j.returncode == 0, err[-4000:]
    r = subprocess.run([CLANG, "-o", exe, *objects], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


@pytest.mark.skipif(CLANG is None, reason="clang++ not available")
@pytest.mark.parametrize("rules", [{}, LARGE], ids=["small", "large"])
def test_linattn_cpu(tmp_path, rules):
    exe = build(str(tmp_path), rules)
    runs = [subprocess.Popen([exe, side], stdout=subprocess.PIPE, text=True) for side in ("front", "back")]
    for r in runs:
        out, _ = r.communicate(timeout=900)
        print(out[-6000:])
        assert r.returncode == 0 and "linattn ok" in out, f"{r.returncode}\n{out[-3000:]}"
