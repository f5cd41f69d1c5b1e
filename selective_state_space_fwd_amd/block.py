"""The operators around the scan in a Mamba block: the short causal convolution before it, the
single-token steps against a cache of request states, and the gated RMS norm after it.

Argument marshalling only, over the C ABI of include/ssm_conv.h, ssm_step.h and ssm_norm.h. The
package exports every function here.

    out, final_state = conv(x, weight, bias=None, silu=False, initial_state=None, lengths=None)
    grads = conv_backward(x, weight, dout, bias=None, silu=False, initial_state=None,
                          lengths=None, dfinal=None)
    out, final_state = causal_conv(...as conv...)                 # differentiable
    out = conv_step(x, state, weight, bias=None, silu=False, slots=None)
    out = scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None,
                    delta_softplus=False, slots=None)             # Mamba-1
    out = ssd_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=False,
                   slots=None)                                    # Mamba-2
    out = norm(y, weight, z=None, eps=1e-5, groups=1, norm_before_gate=False,
               token_major=False)
    out, rstd = norm_train(...as norm...)
    grads = norm_backward(y, weight, rstd, dout, z=None, groups=1, norm_before_gate=False,
                          token_major=False)
    out = gated_norm(...as norm...)                               # differentiable

Tensors of [batch, dim, seqlen] values (x, y, z) may be views with either the steps or the
channels contiguous: the scan's output, or ``proj[:, :, a:b].transpose(1, 2)`` of a
token-major projection. Both are read in place; any other view is copied first. The calls run
on the current stream of the tensors' device, whichever device is current.
"""
from __future__ import annotations

import ctypes
import os
import warnings
from typing import Dict, Optional, Tuple

from . import (SSM_DELTA_SOFTPLUS, SSM_ERR_UNSUPPORTED, SSM_IO_BF16, SSM_IO_F32, SSM_OK,
               SsmScanError, _ptr, lib)
from .build import BINDING_PATH

SSM_CONV_SILU = 1 << 11
SSM_NORM_BEFORE_GATE = 1 << 12

_Strides = ctypes.c_int64 * 3
_bound = _binding = None


class _NoModule:
    """In the place of the extension module where none was built: it makes no call, so that the
    checks below make every one."""

    @staticmethod
    def _makes_none(*args):
        return None

    conv = conv_step = state_step = norm = conv_backward = norm_backward = _makes_none
    bind_linattn = linattn = linattn_backward = linattn_step = _makes_none
    qk_norm = qk_norm_backward = _makes_none


def _lib() -> ctypes.CDLL:
    """libssmscan.so with the argument types of the entry points below, and the extension module
    (csrc/binding.cpp) given their addresses."""
    global _bound, _binding
    if _bound is not None:
        return _bound
    L = lib()
    vp, i64, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32
    L.ssm_conv_fwd.argtypes = [vp, vp, vp, vp, vp, vp, u32, vp, vp, i64, i64, i64, i64, vp]
    L.ssm_conv_bwd.argtypes = [vp, vp, vp, vp, vp, vp, u32, vp, vp, vp, vp, vp, vp, vp, vp,
                               i64, i64, i64, i64, i64, vp]
    L.ssm_conv_bwd_workspace_bytes.argtypes = [i64, i64, i64, i64, u32]
    L.ssm_conv_step.argtypes = [vp, i64, vp, vp, vp, vp, u32, vp, i64, i64, i64, i64, vp]
    L.ssm_scan_step.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp, vp,
                                u32, vp, vp, i64, i64, i64, i64, vp]
    L.ssm_ssd_step.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp, vp,
                               u32, vp, vp, i64, i64, i64, i64, i64, vp]
    L.ssm_norm_fwd.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, u32, vp, vp, vp, vp, i64, i64,
                               i64, i64, i64, vp]
    L.ssm_norm_fwd_workspace_bytes.argtypes = [i64, i64, i64, i64, u32]
    L.ssm_norm_fwd_workspace_bytes.restype = i64
    L.ssm_norm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, u32, vp, vp, vp, vp, vp, vp,
                               i64, i64, i64, i64, i64, vp]
    L.ssm_norm_bwd_workspace_bytes.argtypes = [i64, i64, i64, i64, u32]
    for name in ("ssm_conv_fwd", "ssm_conv_bwd", "ssm_conv_step", "ssm_scan_step",
                 "ssm_ssd_step", "ssm_norm_fwd", "ssm_norm_bwd"):
        getattr(L, name).restype = ctypes.c_int
    L.ssm_conv_bwd_workspace_bytes.restype = i64
    L.ssm_norm_bwd_workspace_bytes.restype = i64
    if not os.path.exists(BINDING_PATH):
        warnings.warn(f"{BINDING_PATH} is missing (python -m selective_state_space_fwd_amd.build): "
                      "every call is marshalled in Python, a few microseconds more each")
        _binding = _NoModule
        _bound = L
        return L
    from . import _binding as module

    address = lambda name: ctypes.cast(getattr(L, name), vp).value
    module.bind(*map(address, ("ssm_conv_fwd", "ssm_conv_step", "ssm_scan_step", "ssm_ssd_step",
                               "ssm_norm_fwd", "ssm_conv_bwd", "ssm_conv_bwd_workspace_bytes",
                               "ssm_norm_bwd", "ssm_norm_bwd_workspace_bytes",
                               "ssm_norm_fwd_workspace_bytes")), SsmScanError)
    _binding = module
    _bound = L
    return L


def _load():
    """The extension module, on first use."""
    _torch()
    _lib()
    return _binding


# ------------------------------------------------------------------ raw C entry points

def ssm_conv_fwd(*args) -> int:
    return _lib().ssm_conv_fwd(*args)


def ssm_conv_bwd(*args) -> int:
    return _lib().ssm_conv_bwd(*args)


def ssm_conv_bwd_workspace_bytes(batch, dim, width, seqlen, flags) -> int:
    return _lib().ssm_conv_bwd_workspace_bytes(batch, dim, width, seqlen, flags)


def ssm_conv_step(*args) -> int:
    return _lib().ssm_conv_step(*args)


def ssm_scan_step(*args) -> int:
    return _lib().ssm_scan_step(*args)


def ssm_ssd_step(*args) -> int:
    return _lib().ssm_ssd_step(*args)


def ssm_norm_fwd(*args) -> int:
    return _lib().ssm_norm_fwd(*args)


def ssm_norm_fwd_workspace_bytes(batch, dim, groups, seqlen, flags) -> int:
    return _lib().ssm_norm_fwd_workspace_bytes(batch, dim, groups, seqlen, flags)


def ssm_norm_bwd(*args) -> int:
    return _lib().ssm_norm_bwd(*args)


def ssm_norm_bwd_workspace_bytes(batch, dim, groups, seqlen, flags) -> int:
    return _lib().ssm_norm_bwd_workspace_bytes(batch, dim, groups, seqlen, flags)


# ------------------------------------------------------------------ checks and the call
#
# A decode loop makes these calls once per layer and token. Where every argument is what the C
# ABI takes as it stands, the functions below go through csrc/binding.cpp, which looks at them in
# C++ and returns None, having done nothing, when one is not; the checks here then copy what
# needs copying and name what is wrong. (conv_step of 8 rows: 4.5 us a call there, 8.4 here, of
# which the launch is 3; ssd_step 5.0 and 11.6.)

def _io_flag(name, t) -> int:
    dtype = t.dtype
    if dtype is _torch().bfloat16:
        return SSM_IO_BF16
    if dtype is _torch().float32:
        return SSM_IO_F32
    raise TypeError(f"unsupported storage dtype {dtype} of {name}")


def _check(name, t, shape, dtype, dev):
    """t has this shape and dtype and is on device number dev."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be on cuda:{dev}")


def _check_out(name, t, shape, dtype, dev):
    _check(name, t, shape, dtype, dev)
    if not t.is_contiguous() or t.is_neg():
        raise ValueError(f"{name} must be contiguous")


def _param(name, t, shape, dtype, dev):
    """An optional array that the C ABI takes contiguous (a strided one is copied)."""
    if t is None:
        return None
    _check(name, t, shape, dtype, dev)
    return t.resolve_neg().contiguous()


def _device(name, t) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


_torch_module = _raw_stream = _current_device = None


def _torch():
    """torch, imported on first use; with it, the cheapest ways to its current stream's handle
    and device number that it offers."""
    global _torch_module, _raw_stream, _current_device
    if _torch_module is None:
        import torch

        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch_module = torch
    return _torch_module


def _run(fn, dev, *args):
    """fn(*args, stream) on the current stream of device `dev`, with that device current."""
    if _current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with _torch().cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status != SSM_OK:
        raise SsmScanError(status)


def _wrote(*tensors):
    """A call wrote these (or None) in place: autograd, if it holds one for a backward pass, has to
    see that."""
    for t in tensors:
        if t is not None and not t.is_inference():
            _torch().autograd.graph.increment_version(t)


def _in_place(t):
    """t, or a contiguous copy of a view with neither steps nor channels contiguous."""
    t = t.resolve_neg()  # (its memory may hold the negative of its values)
    b, d, L = t.shape
    return t if L <= 1 or t.stride(2) == 1 or (d > 1 and t.stride(1) == 1) else t.contiguous()


def _rows(t):
    """t, or a copy with its last axis contiguous."""
    t = t.resolve_neg()
    return t if t.stride(1) == 1 or t.shape[1] <= 1 else t.contiguous()


def _strides(t):
    return _Strides(*t.stride())


def _empty_like_order(t):
    """An uninitialised tensor of t's shape with t's contiguous axis (dense)."""
    b, d, L = t.shape
    if L <= 1 or t.stride(2) == 1:
        return t.new_empty((b, d, L))
    return t.new_empty((b, L, d)).transpose(1, 2)


def _workspace(workspace, need, like):
    torch = _torch()
    if need < 0:
        raise SsmScanError(SSM_ERR_UNSUPPORTED)
    if workspace is None:
        return like.new_empty((max(need, 1),), dtype=torch.uint8)
    if (workspace.dtype != torch.uint8 or workspace.get_device() != like.get_device()
            or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace


# ------------------------------------------------------------------ the short convolution

def _conv_inputs(x, weight, bias, initial_state, lengths):
    torch = _torch()
    dev = _device("x", x)
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [batch, dim, seqlen] and weight [dim, width]")
    flags, f32 = _io_flag("x", x), torch.float32
    batch, dim, seqlen = x.shape
    width = weight.shape[1]
    return (flags, dev, _in_place(x), _param("weight", weight, (dim, width), f32, dev),
            _param("bias", bias, (dim,), f32, dev),
            _param("initial_state", initial_state, (batch, dim, width - 1), x.dtype, dev),
            _param("lengths", lengths, (batch,), torch.int32, dev), batch, dim, width, seqlen)


def conv(x, weight, bias=None, silu: bool = False, initial_state=None, lengths=None, out=None,
         final_state=None, return_final_state: bool = True
         ) -> Tuple["torch.Tensor", Optional["torch.Tensor"]]:
    """Causal depthwise convolution over the last ``width`` (2, 3 or 4) steps.

    x: [batch, dim, seqlen] float32 or bfloat16, steps or channels contiguous; weight: [dim,
    width], bias: [dim] (float32); silu: out = p sigmoid(p); initial_state: [batch, dim,
    width-1], the inputs before the first step, oldest first (None: zero); lengths: [batch]
    int32, the steps of each row (clamped to [0, seqlen]; behind them out is 0 and x is not
    read). Returns (out [batch, dim, seqlen] contiguous, final_state [batch, dim, width-1]: the
    last inputs of each row, the initial_state of a next call), in x's dtype.
    """
    r = (_binding or _load()).conv(x, weight, bias, silu, initial_state, lengths, out, final_state,
                                   return_final_state)
    if r is not None:
        return r
    (flags, dev, x, weight, bias, initial_state, lengths, batch, dim, width,
     seqlen) = _conv_inputs(x, weight, bias, initial_state, lengths)
    if out is None:
        out = x.new_empty((batch, dim, seqlen))
    else:
        _check_out("out", out, (batch, dim, seqlen), x.dtype, dev)
    if final_state is not None:
        _check_out("final_state", final_state, (batch, dim, width - 1), x.dtype, dev)
    elif return_final_state:
        final_state = x.new_empty((batch, dim, max(width - 1, 0)))
    _run(_lib().ssm_conv_fwd, dev, x.data_ptr(), _strides(x), weight.data_ptr(), _ptr(bias),
         _ptr(initial_state), _ptr(lengths), flags | (SSM_CONV_SILU if silu else 0),
         out.data_ptr(), _ptr(final_state), batch, dim, width, seqlen)
    _wrote(out, final_state)
    return out, final_state


def conv_backward(x, weight, dout, bias=None, silu: bool = False, initial_state=None,
                  lengths=None, dfinal=None, want_dinitial: Optional[bool] = None,
                  workspace=None) -> Dict[str, Optional["torch.Tensor"]]:
    """Gradients of sum(dout * out) + sum(dfinal * final_state) for ``conv`` on the same
    inputs: dx (x's dtype and contiguous axis), dweight and dbias (float32; dbias None without
    a bias), dinitial (x's dtype; by default where an initial_state is given, None else).
    Bitwise reproducible. workspace: a uint8 device tensor of at least
    ssm_conv_bwd_workspace_bytes(...) bytes, allocated here when None."""
    r = (_binding or _load()).conv_backward(x, weight, dout, bias, silu, initial_state, lengths,
                                            dfinal, want_dinitial, workspace)
    if r is not None:
        return dict(zip(("dx", "dweight", "dbias", "dinitial"), r))
    f32 = _torch().float32
    (flags, dev, x, weight, bias, initial_state, lengths, batch, dim, width,
     seqlen) = _conv_inputs(x, weight, bias, initial_state, lengths)
    io = x.dtype
    dout = _param("dout", dout, (batch, dim, seqlen), io, dev)
    dfinal = _param("dfinal", dfinal, (batch, dim, width - 1), io, dev)
    if want_dinitial is None:
        want_dinitial = initial_state is not None
    flags |= SSM_CONV_SILU if silu else 0
    workspace = _workspace(
        workspace, _lib().ssm_conv_bwd_workspace_bytes(batch, dim, width, seqlen, flags), x)
    g = {"dx": _empty_like_order(x), "dweight": x.new_empty((dim, width), dtype=f32),
         "dbias": None if bias is None else x.new_empty((dim,), dtype=f32),
         "dinitial": x.new_empty((batch, dim, width - 1)) if want_dinitial else None}
    _run(_lib().ssm_conv_bwd, dev, x.data_ptr(), _strides(x), weight.data_ptr(), _ptr(bias),
         _ptr(initial_state), _ptr(lengths), flags, dout.data_ptr(), _ptr(dfinal),
         g["dx"].data_ptr(), _strides(g["dx"]), g["dweight"].data_ptr(), _ptr(g["dbias"]),
         _ptr(g["dinitial"]), workspace.data_ptr(), workspace.numel(), batch, dim, width, seqlen)
    return g


def conv_step(x, state, weight, bias=None, silu: bool = False, slots=None, out=None):
    """One token of ``conv`` for a batch of requests against a cache of their past inputs.

    x: [batch, dim] (channels contiguous, any row stride); state: [nslots, dim, width-1]
    contiguous, x's dtype, updated in place; slots: [batch] int32, the slot of each row (None:
    row i is slot i). A row whose slot lies outside [0, nslots) gives 0 and changes nothing;
    rows naming one slot are successive tokens of it. Returns out [batch, dim]."""
    r = (_binding or _load()).conv_step(x, state, weight, bias, silu, slots, out)
    if r is not None:
        return r
    torch = _torch()
    dev = _device("x", x)
    if x.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [batch, dim] and state [nslots, dim, width - 1]")
    flags, io, f32 = _io_flag("x", x), x.dtype, torch.float32
    batch, dim = x.shape
    nslots, _, past = state.shape
    _check_out("state", state, (nslots, dim, past), io, dev)
    weight = _param("weight", weight, (dim, past + 1), f32, dev)
    bias = _param("bias", bias, (dim,), f32, dev)
    slots = _param("slots", slots, (batch,), torch.int32, dev)
    x = _rows(x)
    if out is None:
        out = x.new_empty((batch, dim))
    else:
        _check_out("out", out, (batch, dim), io, dev)
    _run(_lib().ssm_conv_step, dev, x.data_ptr(), x.stride(0), state.data_ptr(),
         weight.data_ptr(), _ptr(bias), _ptr(slots), flags | (SSM_CONV_SILU if silu else 0),
         out.data_ptr(), batch, nslots, dim, past + 1)
    _wrote(state, out)
    return out


# ------------------------------------------------------------------ the state step

def _step(fn, heads, x, dt, A, B, C, state, D, z, dt_bias, softplus, slots, out, names):
    torch = _torch()
    dev = _device(names[0], x)
    if x.dim() != 2 or state.dim() != 3 or B.dim() != 2:
        raise ValueError(f"{names[0]} must be [batch, dim], B and C [batch, dstate] and state "
                         "[nslots, dim, dstate]")
    flags, io, f32 = _io_flag(names[0], x), x.dtype, torch.float32
    batch, dim = x.shape
    nslots, _, dstate = state.shape
    steps = dim if heads is None else heads
    _check_out("state", state, (nslots, dim, dstate), f32, dev)
    _check(names[1], dt, (batch, steps), io, dev)
    _check("B", B, (batch, dstate), io, dev)
    _check("C", C, (batch, dstate), io, dev)
    A = _param("A", A, (dim, dstate) if heads is None else (heads,), f32, dev)
    D = _param("D", D, (dim,), f32, dev)
    dt_bias = _param(names[2], dt_bias, (steps,), f32, dev)
    slots = _param("slots", slots, (batch,), torch.int32, dev)
    z_ptr = z_stride = 0
    if z is not None:
        _check("z", z, (batch, dim), io, dev)
        z = _rows(z)
        z_ptr, z_stride = z.data_ptr(), z.stride(0)
    x, dt, B, C = _rows(x), _rows(dt), _rows(B), _rows(C)
    if out is None:
        out = x.new_empty((batch, dim))
    else:
        _check_out("out", out, (batch, dim), io, dev)
    sizes = (dim,) if heads is None else (heads, dim // heads)
    _run(fn, dev, x.data_ptr(), x.stride(0), dt.data_ptr(), dt.stride(0), A.data_ptr(),
         B.data_ptr(), B.stride(0), C.data_ptr(), C.stride(0), _ptr(D), z_ptr, z_stride,
         _ptr(dt_bias), _ptr(slots), flags | (SSM_DELTA_SOFTPLUS if softplus else 0),
         state.data_ptr(), out.data_ptr(), batch, nslots, *sizes, dstate)
    _wrote(state, out)
    return out


def scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None,
              delta_softplus: bool = False, slots=None, out=None):
    """One token of the selective scan for a batch of requests against a cache of states.

    u, delta, z: [batch, dim]; B, C: [batch, dstate] (float32 or bfloat16, any row stride);
    A: [dim, dstate], D and delta_bias: [dim] (float32); state: [nslots, dim, dstate] float32
    contiguous, updated in place (dstate at most 256); slots: [batch] int32, the slot of each
    row (None: row i is slot i). A row whose slot lies outside [0, nslots) gives 0 and changes
    nothing; rows naming one slot are successive tokens of it. Returns out [batch, dim]."""
    r = (_binding or _load()).state_step(False, u, delta, A, B, C, state, D, z, delta_bias,
                                         delta_softplus, slots, out)
    if r is not None:
        return r
    if A.dim() != 2:
        raise ValueError("A must be [dim, dstate]")
    return _step(_lib().ssm_scan_step, None, u, delta, A, B, C, state, D, z, delta_bias,
                 delta_softplus, slots, out, ("u", "delta", "delta_bias"))


def ssd_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
             slots=None, out=None):
    """One token of the Mamba-2 recurrence (``ssd``), as ``scan_step``: x, z: [batch,
    nheads*headdim]; dt: [batch, nheads]; A, dt_bias: [nheads]; D: [nheads*headdim]."""
    r = (_binding or _load()).state_step(True, x, dt, A, B, C, state, D, z, dt_bias, dt_softplus,
                                         slots, out)
    if r is not None:
        return r
    if A.dim() != 1:
        raise ValueError("A must be [nheads]")
    heads = A.shape[0]
    if heads == 0 or x.dim() != 2 or x.shape[1] % heads:
        raise ValueError("x must be [batch, channels], the channels a multiple of the head count")
    return _step(_lib().ssm_ssd_step, heads, x, dt, A, B, C, state, D, z, dt_bias, dt_softplus,
                 slots, out, ("x", "dt", "dt_bias"))


# ------------------------------------------------------------------ the gated norm

def _norm_inputs(y, weight, z, groups):
    dev = _device("y", y)
    if y.dim() != 3:
        raise ValueError("y must be [batch, dim, seqlen]")
    flags = _io_flag("y", y)
    batch, dim, seqlen = y.shape
    if groups < 1 or dim % groups:
        raise ValueError("the channel count must be a multiple of groups")
    weight = _param("weight", weight, (dim,), _torch().float32, dev)
    if z is not None:
        _check("z", z, y.shape, y.dtype, dev)
        z = _in_place(z)
    return flags, dev, _in_place(y), z, weight, batch, dim, seqlen


def _norm_forward(y, weight, z, eps, groups, norm_before_gate, token_major, out, save):
    r = (_binding or _load()).norm(y, weight, z, eps, groups, norm_before_gate, token_major, out,
                                   save)
    if r is not None:
        return r
    flags, dev, y, z, weight, batch, dim, seqlen = _norm_inputs(y, weight, z, groups)
    shape = (batch, seqlen, dim) if token_major else (batch, dim, seqlen)
    if out is None:
        out = y.new_empty(shape)
    else:
        _check_out("out", out, shape, y.dtype, dev)
    rstd = y.new_empty((batch, groups, seqlen), dtype=_torch().float32) if save else None
    z_ptr = z_strides = None
    if z is not None:
        z_ptr, z_strides = z.data_ptr(), _strides(z)
    workspace = _workspace(
        None, _lib().ssm_norm_fwd_workspace_bytes(batch, dim, groups, seqlen, flags), y)
    _run(_lib().ssm_norm_fwd, dev, y.data_ptr(), _strides(y), z_ptr, z_strides,
         weight.data_ptr(), eps, flags | (SSM_NORM_BEFORE_GATE if norm_before_gate else 0),
         out.data_ptr(), _Strides(seqlen * dim, 1, dim) if token_major else None, _ptr(rstd),
         workspace.data_ptr(), workspace.numel(), batch, dim, groups, seqlen)
    _wrote(out)
    return out, rstd


def norm(y, weight, z=None, eps: float = 1e-5, groups: int = 1, norm_before_gate: bool = False,
         token_major: bool = False, out=None):
    """RMS norm over the channels of each of ``groups`` equal groups, with a gate.

    y, z: [batch, dim, seqlen] float32 or bfloat16, steps or channels contiguous; weight: [dim]
    float32. out = weight v / sqrt(mean(v^2) + eps) with v = y silu(z), or, with
    norm_before_gate, v = y and the result times silu(z); z None: no gate. Returns out in y's
    dtype, contiguous: [batch, dim, seqlen], or [batch, seqlen, dim] with token_major (the
    order an output projection reads)."""
    return _norm_forward(y, weight, z, eps, groups, norm_before_gate, token_major, out, False)[0]


def norm_train(y, weight, z=None, eps: float = 1e-5, groups: int = 1,
               norm_before_gate: bool = False, token_major: bool = False, out=None):
    """``norm`` that also returns 1 / sqrt(mean + eps) of every token and group, [batch,
    groups, seqlen] float32, which ``norm_backward`` takes."""
    return _norm_forward(y, weight, z, eps, groups, norm_before_gate, token_major, out, True)


def norm_backward(y, weight, rstd, dout, z=None, groups: int = 1, norm_before_gate: bool = False,
                  token_major: bool = False, workspace=None
                  ) -> Dict[str, Optional["torch.Tensor"]]:
    """Gradients of sum(dout * out) for ``norm`` on the same inputs: dy, dz (y's dtype, each with
    its input's contiguous axis; dz None without a gate) and dweight (float32). rstd:
    ``norm_train``'s; dout: of out's shape, steps or channels contiguous. Bitwise
    reproducible. workspace: a uint8 device tensor of at least
    ssm_norm_bwd_workspace_bytes(...) bytes, allocated here when None."""
    r = (_binding or _load()).norm_backward(y, weight, rstd, dout, z, groups, norm_before_gate,
                                            token_major, workspace)
    if r is not None:
        return dict(zip(("dy", "dz", "dweight"), r))
    f32 = _torch().float32
    flags, dev, y, z, weight, batch, dim, seqlen = _norm_inputs(y, weight, z, groups)
    _check_out("rstd", rstd, (batch, groups, seqlen), f32, dev)
    _check("dout", dout, (batch, seqlen, dim) if token_major else (batch, dim, seqlen), y.dtype,
           dev)
    dout = _in_place(dout.transpose(1, 2) if token_major else dout)
    flags |= SSM_NORM_BEFORE_GATE if norm_before_gate else 0
    workspace = _workspace(
        workspace, _lib().ssm_norm_bwd_workspace_bytes(batch, dim, groups, seqlen, flags), y)
    g = {"dy": _empty_like_order(y), "dz": None if z is None else _empty_like_order(z),
         "dweight": y.new_empty((dim,), dtype=f32)}
    _run(_lib().ssm_norm_bwd, dev, y.data_ptr(), _strides(y), _ptr(z),
         None if z is None else _strides(z), weight.data_ptr(), rstd.data_ptr(), dout.data_ptr(),
         _strides(dout), flags, g["dy"].data_ptr(), _strides(g["dy"]), _ptr(g["dz"]),
         None if z is None else _strides(g["dz"]), g["dweight"].data_ptr(), workspace.data_ptr(),
         workspace.numel(), batch, dim, groups, seqlen)
    return g


# ------------------------------------------------------------------ autograd

_functions = None


def _autograd():
    """The torch.autograd.Functions behind ``causal_conv`` and ``gated_norm`` (built on first
    use, so that importing this module does not import torch)."""
    global _functions
    if _functions is not None:
        return _functions
    import torch
    from torch.autograd.function import once_differentiable

    class CausalConv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, initial_state, lengths, silu):
            out, fin = conv(x, weight, bias=bias, silu=silu, initial_state=initial_state,
                            lengths=lengths)
            ctx.save_for_backward(x, weight, bias, initial_state, lengths)
            ctx.silu = silu
            ctx.set_materialize_grads(False)
            return out, fin

        @staticmethod
        @once_differentiable
        def backward(ctx, dout, dfin):
            x, weight, bias, initial_state, lengths = ctx.saved_tensors
            dout = x.new_zeros(x.shape) if dout is None else dout
            g = conv_backward(x, weight, dout, bias=bias, silu=ctx.silu,
                              initial_state=initial_state, lengths=lengths, dfinal=dfin)
            return g["dx"], g["dweight"], g["dbias"], g["dinitial"], None, None

    class GatedNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, weight, z, eps, groups, norm_before_gate, token_major):
            out, rstd = norm_train(y, weight, z=z, eps=eps, groups=groups,
                                   norm_before_gate=norm_before_gate, token_major=token_major)
            ctx.save_for_backward(y, weight, z, rstd)
            ctx.options = dict(groups=groups, norm_before_gate=norm_before_gate,
                               token_major=token_major)
            return out

        @staticmethod
        @once_differentiable
        def backward(ctx, dout):
            y, weight, z, rstd = ctx.saved_tensors
            g = norm_backward(y, weight, rstd, dout, z=z, **ctx.options)
            return g["dy"], g["dweight"], g["dz"], None, None, None, None

    _functions = (CausalConv, GatedNorm)
    return _functions


def causal_conv(x, weight, bias=None, silu: bool = False, initial_state=None, lengths=None
                ) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """Differentiable ``conv``: (out, final_state), with gradients for x, weight, bias and
    initial_state through autograd (``conv_backward``)."""
    return _autograd()[0].apply(x, weight, bias, initial_state, lengths, bool(silu))


def gated_norm(y, weight, z=None, eps: float = 1e-5, groups: int = 1,
               norm_before_gate: bool = False, token_major: bool = False) -> "torch.Tensor":
    """Differentiable ``norm``, with gradients for y, weight and z through autograd
    (``norm_backward``)."""
    return _autograd()[1].apply(y, weight, z, float(eps), int(groups), bool(norm_before_gate),
                                bool(token_major))
