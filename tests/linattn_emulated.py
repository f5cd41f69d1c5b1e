"""The linear-attention kernels and those of the queries' and keys' norm in a CPU build
(tests/host/emulate_mma), as a shared library called through the C ABI with numpy arrays."""
import ctypes
import os
import re
import subprocess
import tempfile

import numpy as np

import selective_state_space_fwd_amd as ssm
from test_linattn_cpu import CLANG, CSRC, HERE, HOST, KERNELS, ROOT

HEADERS = ("device_block.h", "device_linattn.h", "linattn_launch.h", "qk_launch.h", "heads.h")


_built = {}  # by launch rules: (the library, its folder), for all test files of a process


def kernels_of(rules):
    """The library with these launch rules in place of the headers'."""
    key = tuple(sorted(rules.items()))
    if key not in _built:
        folder = tempfile.TemporaryDirectory(prefix="linattn")
        _built[key] = build(folder.name, rules), folder
    return _built[key][0]


def build(folder, rules):
    found = set()
    for name in (*KERNELS, *HOST, *HEADERS):  # copies: their includes find the CPU's device_math.h and device_scan.h
        text = open(os.path.join(CSRC, name)).read()
        for rule, value in rules.items():
            text, n = re.subn(rf"(constexpr int64_t {rule} =)[^;]*;", rf"\1 {value};", text)
            found |= {rule} if n else set()
        text = re.sub(r'asm volatile\("s_waitcnt[^;]*;', "__syncthreads();", text)
        text = text.replace("__attribute__((address_space(3)))", "")
        with open(os.path.join(folder, name.replace(".hip", ".cpp")), "w") as f:
            f.write(text)
    assert found == set(rules)
    flags = [CLANG, "-std=c++20", "-O1", "-fno-unroll-loops", "-fPIC", "-Wno-everything", "-I",
             os.path.join(HERE, "host", "emulate_mma"), "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    sources = [os.path.join(folder, k.replace(".hip", ".cpp")) for k in (*HOST, *KERNELS)]
    objects = [s + ".o" for s in sources]
    jobs = [subprocess.Popen([*flags, "-c", s, "-o", o], stderr=subprocess.PIPE, text=True)
            for s, o in zip(sources, objects)]
    for j in jobs:
        _, err = j.communicate()
        assert j.returncode == 0, err[-4000:]
    target = os.path.join(folder, "liblinattn_cpu.so")
    r = subprocess.run([CLANG, "-shared", "-o", target, *objects], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return Emulated(target)


def rounded(x, io):
    """The values of x in the storage type, as float64."""
    x = np.asarray(x, np.float32)
    if io == "f32":
        return x.astype(np.float64)
    u = x.view(np.uint32).astype(np.uint64)
    return (((u + 0x7fff + (u >> 16 & 1)) >> 16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def stored(x, io):
    """An array of the storage type with these values (bf16 as its bits)."""
    x = np.ascontiguousarray(x, np.float32)
    return x if io == "f32" else (x.view(np.uint32) >> 16).astype(np.uint16)


def widened(x):
    return ((x.astype(np.uint32) << 16).view(np.float32) if x.dtype == np.uint16 else x).astype(np.float64)


def pointer(x):
    return None if x is None else x.ctypes.data_as(ctypes.c_void_p)


def empty(shape, io="f32"):
    return np.full(shape, 7, np.float32 if io == "f32" else np.uint16)


class Emulated:
    """Inputs as float64 values that their storage type holds, results as float64."""

    def __init__(self, path):
        self.lib = L = ctypes.CDLL(path)
        vp, i64, u32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
        L.ssm_linattn_fwd.argtypes = [vp] * 10 + [f32, u32, vp, vp, vp] + [i64] * 7 + [vp]
        L.ssm_linattn_bwd.argtypes = [vp] * 13 + [f32, u32] + [vp] * 6 + [i64] * 7 + [vp]
        L.ssm_qk_norm_fwd.argtypes = [vp] * 9 + [f32, u32, vp, vp] + [i64] * 7 + [vp]
        L.ssm_qk_norm_bwd.argtypes = [vp] * 13 + [f32, u32] + [vp] * 5 + [i64] * 8 + [vp]
        for name in ("ssm_linattn_fwd_workspace_bytes", "ssm_linattn_bwd_workspace_bytes"):
            getattr(L, name).argtypes, getattr(L, name).restype = [i64] * 5 + [u32], i64
        L.ssm_qk_norm_bwd_workspace_bytes.argtypes = [i64] * 6 + [u32]
        L.ssm_qk_norm_bwd_workspace_bytes.restype = i64

    @staticmethod
    def _workspace(n):
        ws = np.full(n + 256, 0xff, np.uint8)
        return ws, ctypes.c_void_p((ws.ctypes.data + 255) // 256 * 256)

    @staticmethod
    def _inputs(io, q, k, v, g, initial_state, lengths):
        b, L, hk, dk = q.shape
        h, dv = v.shape[2:]
        per_head = g is not None and g.ndim == 1
        f32 = lambda x: None if x is None else np.ascontiguousarray(x, np.float32)
        n = None if lengths is None else np.asarray(lengths, np.int32)
        strides = (ctypes.c_int64 * 3)(0, 0, 1) if per_head else None
        arrays = (stored(q, io), stored(k, io), stored(v, io), f32(g), f32(initial_state), n)
        return arrays, strides, per_head, (b, L, hk, h, dk, dv), ssm.SSM_IO_F32 if io == "f32" else ssm.SSM_IO_BF16

    def forward(self, io, q, k, v, g=None, initial_state=None, lengths=None):
        (q, k, v, g, s0, n), gs, _, (b, L, hk, h, dk, dv), flags = self._inputs(io, q, k, v, g, initial_state, lengths)
        need = self.lib.ssm_linattn_fwd_workspace_bytes(b, L, h, dk, dv, flags)
        ws, at = self._workspace(need)
        out, fin = empty((b, L, h, dv), io), empty((b, h, dv, dk))
        status = self.lib.ssm_linattn_fwd(
            pointer(q), None, pointer(k), None, pointer(v), None, pointer(g), gs, pointer(s0), pointer(n), dk ** -0.5,
            flags, pointer(out), pointer(fin), at, need, b, L, hk, h, dk, dv, None)
        assert status == ssm.SSM_OK
        return widened(out), widened(fin)

    def backward(self, io, q, k, v, dout, g=None, initial_state=None, lengths=None, dfinal=None):
        (q, k, v, g, s0, n), gs, per_head, (b, L, hk, h, dk, dv), flags = self._inputs(
            io, q, k, v, g, initial_state, lengths)
        flags |= ssm.SSM_LINATTN_HEAD_DG if per_head else 0
        need = self.lib.ssm_linattn_bwd_workspace_bytes(b, L, h, dk, dv, flags)
        ws, at = self._workspace(need)
        dout = stored(dout, io)
        ds = None if dfinal is None else np.ascontiguousarray(dfinal, np.float32)
        d = {"dq": empty((b, L, hk, dk), io), "dk": empty((b, L, hk, dk), io), "dv": empty((b, L, h, dv), io),
             "dg": None if g is None else empty(g.shape), "dinitial": empty((b, h, dv, dk))}
        status = self.lib.ssm_linattn_bwd(
            pointer(q), None, pointer(k), None, pointer(v), None, pointer(dout), None, pointer(g), gs, pointer(s0),
            pointer(n), pointer(ds), dk ** -0.5, flags, *(pointer(x) for x in d.values()), at, need, b, L, hk, h, dk,
            dv, None)
        assert status == ssm.SSM_OK
        return {name: None if x is None else widened(x) for name, x in d.items()}

    def qk(self, io, q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, eps=1e-6):
        """(q_out, k_out, dq, dk, dq_weight, dk_weight); cos and sin may be None."""
        b, L, hq, d = q.shape
        hk, rows, rot = k.shape[2], 0 if cos is None else len(cos), 0 if cos is None else 2 * cos.shape[1]
        flags = ssm.SSM_IO_F32 if io == "f32" else ssm.SSM_IO_BF16
        f32 = lambda x: None if x is None else np.ascontiguousarray(x, np.float32)
        q, k, dq_out, dk_out = (stored(x, io) for x in (q, k, dq_out, dk_out))
        shared = [f32(x) for x in (q_weight, k_weight, cos, sin)]
        shared.append(None if positions is None else np.ascontiguousarray(positions, np.int32))
        sizes = (b, L, hq, hk, d, rot, rows)
        qo, ko, dq, dk = empty(q.shape, io), empty(k.shape, io), empty(q.shape, io), empty(k.shape, io)
        qw, kw = empty((d,)), empty((d,))
        status = self.lib.ssm_qk_norm_fwd(pointer(q), None, pointer(k), None, *map(pointer, shared), eps, flags,
                                          pointer(qo), pointer(ko), *sizes, None)
        assert status == ssm.SSM_OK
        need = self.lib.ssm_qk_norm_bwd_workspace_bytes(*sizes[:6], flags)
        ws, at = self._workspace(need)
        status = self.lib.ssm_qk_norm_bwd(
            pointer(q), None, pointer(k), None, pointer(dq_out), None, pointer(dk_out), None, *map(pointer, shared), eps,
            flags, pointer(dq), pointer(dk), pointer(qw), pointer(kw), at, need, *sizes, None)
        assert status == ssm.SSM_OK
        return [widened(x) for x in (qo, ko, dq, dk, qw, kw)]
