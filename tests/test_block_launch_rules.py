"""The launch rules of the operators around the scan (csrc/block_launch.h), on the CPU: which form a
call takes, at the sizes of the tests that compare that form with the oracle and either side of
each rule's edges."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
F32, BF16 = 0, 1

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("rules") / "launch_rules")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(ROOT, "selective_state_space_fwd_amd", "csrc"), "-o", exe,
                        os.path.join(HERE, "host", "launch_rules.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(name, *cases):
        words = [str(int(w)) if not isinstance(w, str) else w for c in cases for w in (name, *c)]
        r = subprocess.run([exe, *words], capture_output=True, text=True)
        assert r.returncode == 0
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return ask


def test_conv_tiles_a_wave(rules):
    """Two only where a row has two: a second tile of a row of at most 512 steps holds nothing, and
    its arithmetic would be done on zeros."""
    two = [(4, 2304, 2048, BF16), (3, 2731, 777, BF16), (2, 2741, 1531, BF16), (1, 4099, 2048, BF16),
           (1, 8192, 513, BF16)]
    one = [(4, 4096, 512, BF16), (16, 6000, 100, BF16), (2, 8200, 500, BF16), (64, 60000, 1, BF16),
           (65535, 32768, 8, BF16), (1, 8191, 513, BF16), (5, 523, 777, BF16), (4, 2304, 2048, F32),
           (1, 1536, 65536, F32), (4, 2304, 0, BF16)]
    assert rules("conv_fwd", *two) == [(2,)] * len(two)
    assert rules("conv_fwd", *one) == [(1,)] * len(one)
