"""Build libssmscan.so in-tree with hipcc for gfx950.

    python -m selective_state_space_fwd_amd.build

Every HIP source is compiled with the packed-fp32 instructions disabled
(-Xclang -target-feature -Xclang -packed-fp32-ops); the host pass warns that it does
not know that feature, which is harmless.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libssmscan.so")
# The VALU throughput probes bench.py --alu-probe runs; a library of their own.
PROBE_SOURCE = os.path.join(PKG, "probes", "alu_probe.hip")
PROBE_LIB_PATH = os.path.join(PKG, "libssmprobe.so")
SOURCES = ["scan_kernels.hip", "scan_short.hip", "scan_bwd.hip", "ssd_kernels.hip", "scan_api.cpp",
           "ssd_api.cpp", "ssd_noalloc.hip", "conv_kernels.hip", "conv_api.cpp", "step_kernels.hip",
           "step_api.cpp", "norm_kernels.hip", "norm_api.cpp"]
# A test-only build of the Mamba-1 scan with a second launch shape of the chunked kernel (the
# same 16 steps per lane, other channels per workgroup and states per LDS stage), which the
# parity tests run against the oracle and against the default build.
SHAPE2_LIB_PATH = os.path.join(PKG, "libssmscan_shape2.so")
SHAPE2_SOURCES = ["scan_kernels.hip", "scan_short.hip", "scan_bwd.hip", "scan_api.cpp"]
SHAPE2_DEFINES = ["-DSSM_BF16_K=4", "-DSSM_BF16_G=4", "-DSSM_F32_K=2", "-DSSM_F32_G=1"]
# The short way from Python into the single-token entry points, an extension module built against
# the installed torch (host code only).
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG, "_binding.so")
ARCH = "gfx950"


def hipcc() -> str:
    return os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def compile_flags() -> list:
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-fvisibility=hidden", "-Wall", "-I", INCLUDE, "-I", CSRC]


def _compile(cmd, sources, target, verbose):
    fd, tmp = tempfile.mkstemp(prefix=os.path.basename(target) + ".", suffix=".tmp", dir=PKG)
    os.close(fd)
    cmd = [*cmd, "-shared", "-o", tmp, *sources]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, cwd=PKG, capture_output=True, text=True)
    if r.returncode != 0:
        os.unlink(tmp)
        raise RuntimeError(f"{cmd[0]} failed ({r.returncode}):\n{r.stderr}")
    umask = os.umask(0)
    os.umask(umask)
    os.chmod(tmp, 0o777 & ~umask)  # (mkstemp's file is its owner's alone, and g++ keeps that)
    os.replace(tmp, target)
    return target


def _link(sources, target, verbose, extra=()):
    return _compile([hipcc(), *compile_flags(), *extra], sources, target, verbose)


def _binding_lacks():
    """What the extension module's build needs and this machine has not, or None."""
    import sysconfig

    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        return f"no C++ compiler ({cxx})"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "no Python.h"
    try:
        from torch.utils.cpp_extension import include_paths
    except ImportError as e:
        return f"no torch ({e})"
    if not any(os.path.exists(os.path.join(p, "ATen", "ATen.h")) for p in include_paths(device_type="cuda")):
        return "no headers of torch"
    return None


def _build_binding(verbose: bool) -> str:
    """_binding.so: g++ against torch's and Python's headers and torch's libraries (found in the
    process by then: the module is imported after torch)."""
    import sysconfig

    from torch.utils.cpp_extension import include_paths, library_paths
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"]]
    for path in include_paths(device_type="cuda"):
        cmd += ["-isystem", path]
    libs = ["-L" + library_paths(device_type="cuda")[0], "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10_hip", "-lc10"]
    return _compile(cmd, [BINDING_SOURCE, *libs], BINDING_PATH, verbose)


def build(verbose: bool = False) -> str:
    """Build libssmprobe.so (the VALU probes), libssmscan_shape2.so (the test-only second launch
    shape), libssmscan.so (the scan library), which hipcc alone makes, and then _binding.so (the
    binding's extension module). Where the last cannot be built for want of a C++ compiler, torch
    or headers, a warning says so and none is left behind: the binding then marshals every call
    in Python."""
    _link([PROBE_SOURCE], PROBE_LIB_PATH, verbose)
    _link([os.path.join(CSRC, s) for s in SHAPE2_SOURCES], SHAPE2_LIB_PATH, verbose,
          SHAPE2_DEFINES)
    _link([os.path.join(CSRC, s) for s in SOURCES], LIB_PATH, verbose)
    lacks = _binding_lacks()
    if lacks is None:
        _build_binding(verbose)
    else:
        if os.path.exists(BINDING_PATH):
            os.unlink(BINDING_PATH)  # of other sources, perhaps
        warnings.warn(f"{os.path.basename(BINDING_PATH)} not built: {lacks}")
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
