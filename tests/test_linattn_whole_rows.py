"""When linear attention loads and stores by words (linattn_launch.h, compiled by the host's compiler): only
where every array of the call, its results among them, lies at 4-byte aligned addresses."""
import shutil
import subprocess

import pytest

from selective_state_space_fwd_amd.build import CSRC, INCLUDE

SOURCE = r"""
#include <stdio.h>
#include "linattn_launch.h"
using namespace ssm;
int main() {
  int bad = 0;
  alignas(16) static char memory[64];
  for (Io io : {Io::BF16, Io::F32}) for (int bwd = 0; bwd < 2; ++bwd) {
    auto args = [&] {
      LinattnArgs a{};
      const HeadRows r{memory, 1024, 256, 64};
      a.q = a.k = a.v = a.dout = r;
      a.out = a.dq = a.dk_ = a.dv_ = memory;
      a.dk = a.dv = 64;
      a.io = io;
      return a;
    };
    bad += !linattn_whole(args(), bwd);
    for (int which = 0; which < 8; ++which) {
      LinattnArgs a = args();
      void* odd = memory + 2;
      const bool used = which < 3 || (which == 4 ? !bwd : bool(bwd));
      if (which == 0) a.q.p = odd;
      if (which == 1) a.k.p = odd;
      if (which == 2) a.v.p = odd;
      if (which == 3) a.dout.p = odd;
      if (which == 4) a.out = odd;
      if (which == 5) a.dq = odd;
      if (which == 6) a.dk_ = odd;
      if (which == 7) a.dv_ = odd;
      if (linattn_whole(a, bwd) == used) printf("io %d bwd %d array %d\n", int(io), bwd, which), ++bad;
    }
    LinattnArgs a = args();
    a.out = a.dq = a.dk_ = a.dv_ = memory + 4;
    bad += !linattn_whole(a, bwd);
  }
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_words_only_where_all_arrays_are_aligned(tmp_path):
    source, exe = tmp_path / "whole.cpp", str(tmp_path / "whole")
    source.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", INCLUDE, "-o", exe, str(source)], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
