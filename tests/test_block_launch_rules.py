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


def test_conv_step_rows_a_lane(rules):
    cases = [(385, 6000, BF16), (385, 6001, F32), (384, 4352, BF16), (70, 2304, F32), (8, 2304, BF16)]
    assert rules("conv_step", *cases) == [(2,), (2,), (2,), (1,), (1,)]


def test_state_step_forms(rules):
    """Channels a lane, and whether the states go past the caches; the last three are of small
    calls."""
    cases = [(256, 2560, 16), (250, 5000, 5), (250, 4099, 7), (40, 4096, 128), (256, 4100, 33), (128, 4096, 64),
             (100, 4096, 100), (200, 6144, 128), (61, 2048, 16), (8, 2048, 128), (3, 5, 1)]
    assert rules("state_step", *cases) == [(4, 0), (2, 0), (2, 0), (8, 0), (8, 1), (8, 1), (8, 1), (8, 1), (2, 0),
                                           (2, 0), (1, 0)]


def test_norm_shapes(rules):
    """(steps, log2 of the lanes along channels, waves, split): the forward's sixteen waves for runs of
    32 bytes, its two launches for odd rows of a result in time order and for groups that do not
    fit; the gradient's eight and sixteen waves and its two launches."""
    order = lambda b, d, L, io, chan, dword: (b, d, 1, L, io, chan, dword)
    fwd = [order(4, 2048, 2047, F32, False, True), order(4, 2048, 2048, F32, False, True),
           order(4, 4096, 1021, BF16, False, False), order(1, 4096, 1023, BF16, False, False),
           order(1, 4096, 1023, BF16, False, True), order(1, 8200, 9, BF16, False, False),
           order(1, 5001, 77, F32, False, True), order(4, 2048, 2048, BF16, False, True),
           order(8, 2048, 1, BF16, True, True)]
    assert rules("norm_fwd", *fwd) == [(4, 5, 16, 0), (4, 5, 16, 0), (8, 5, 16, 0), (8, 3, 4, 1), (8, 6, 8, 0),
                                       (8, 3, 4, 1), (4, 3, 4, 1), (8, 5, 8, 0), (1, 6, 4, 0)]
    bwd = [order(4, 2048, 2048, BF16, False, True), order(4, 2048, 2048, BF16, True, True),
           order(4, 4096, 1021, BF16, False, False), order(1, 2048, 512, BF16, False, True),
           order(4, 2048, 2047, F32, False, True)]
    assert rules("norm_bwd", *bwd) == [(4, 4, 16, 0), (4, 5, 8, 0), (4, 3, 4, 1), (4, 3, 4, 1), (4, 5, 16, 0)]
