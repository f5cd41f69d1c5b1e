"""Linear attention with a decay for each head, and the norm and rotation of the queries and keys
ahead of it.

Argument marshalling only, over the C ABI of include/ssm_linattn.h and ssm_qk.h. The package
exports every function here.

    out, final_state = linattn(q, k, v, g=None, scale=None, initial_state=None, lengths=None)
    grads = linattn_backward(q, k, v, dout, g=None, scale=None, initial_state=None, lengths=None,
                             dfinal=None)
    out, final_state = linear_attention(...as linattn...)          # differentiable
    out = linattn_step(q, k, v, state, g=None, scale=None, slots=None)
    q_out, k_out = qk_norm(q, k, q_weight=None, k_weight=None, cos=None, sin=None,
                           positions=None, eps=1e-6, interleaved=False)
    grads = qk_norm_backward(q, k, dq_out, dk_out, ...as qk_norm...)
    q_out, k_out = rotary_qk_norm(...as qk_norm...)                # differentiable

q and k are [batch, seqlen, qk_heads, dk], v [batch, seqlen, heads, dv], float32 or bfloat16, any
views whose last axis is contiguous: ``proj[..., a:b].unflatten(-1, (heads, dim))`` of a
projection's output is read in place; other views are copied first. The head h of v reads the
query and key head h // (heads // qk_heads). The calls run on the current stream of the tensors'
device, whichever device is current.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional, Tuple

from . import _ptr
from . import block
from .block import (_check, _check_out, _device, _io_flag, _param, _run, _Strides, _torch,
                    _workspace, _wrote)

SSM_LINATTN_HEAD_DG = 1 << 13
SSM_QK_INTERLEAVED = 1 << 14

_bound = _ready = None


def _lib() -> ctypes.CDLL:
    """libssmscan.so with the argument types of the entry points below."""
    global _bound
    if _bound is not None:
        return _bound
    _torch()
    L = block._lib()
    vp, i64, u32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
    L.ssm_linattn_fwd.argtypes = [vp] * 10 + [f32, u32, vp, vp, vp] + [i64] * 7 + [vp]
    L.ssm_linattn_bwd.argtypes = [vp] * 13 + [f32, u32] + [vp] * 6 + [i64] * 7 + [vp]
    L.ssm_linattn_step.argtypes = [vp] * 9 + [f32, u32, vp, vp] + [i64] * 6 + [vp]
    L.ssm_qk_norm_fwd.argtypes = [vp] * 9 + [f32, u32, vp, vp] + [i64] * 7 + [vp]
    L.ssm_qk_norm_bwd.argtypes = [vp] * 13 + [f32, u32] + [vp] * 5 + [i64] * 8 + [vp]
    for name in ("ssm_linattn_fwd_workspace_bytes", "ssm_linattn_bwd_workspace_bytes"):
        getattr(L, name).argtypes = [i64] * 5 + [u32]
        getattr(L, name).restype = i64
    L.ssm_qk_norm_bwd_workspace_bytes.argtypes = [i64] * 6 + [u32]
    L.ssm_qk_norm_bwd_workspace_bytes.restype = i64
    for name in ("ssm_linattn_fwd", "ssm_linattn_bwd", "ssm_linattn_step", "ssm_qk_norm_fwd",
                 "ssm_qk_norm_bwd"):
        getattr(L, name).restype = ctypes.c_int
    _bound = L
    return L


def _native():
    """The extension module (csrc/binding.cpp), given the addresses of the entry points below. Its
    functions make a call whose arguments are what the C ABI takes as they stand, and return None
    without having done anything for any other, which the checks here then take."""
    global _ready
    module = block._binding or block._load()
    if module is not _ready:
        L = _lib()
        module.bind_linattn(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
            "ssm_linattn_fwd", "ssm_linattn_fwd_workspace_bytes", "ssm_linattn_bwd",
            "ssm_linattn_bwd_workspace_bytes", "ssm_linattn_step", "ssm_qk_norm_fwd",
            "ssm_qk_norm_bwd", "ssm_qk_norm_bwd_workspace_bytes")))
        _ready = module
    return module


# ------------------------------------------------------------------ raw C entry points

def ssm_linattn_fwd(*args) -> int:
    return _lib().ssm_linattn_fwd(*args)


def ssm_linattn_fwd_workspace_bytes(batch, seqlen, heads, dk, dv, flags) -> int:
    return _lib().ssm_linattn_fwd_workspace_bytes(batch, seqlen, heads, dk, dv, flags)


def ssm_linattn_bwd(*args) -> int:
    return _lib().ssm_linattn_bwd(*args)


def ssm_linattn_bwd_workspace_bytes(batch, seqlen, heads, dk, dv, flags) -> int:
    return _lib().ssm_linattn_bwd_workspace_bytes(batch, seqlen, heads, dk, dv, flags)


def ssm_linattn_step(*args) -> int:
    return _lib().ssm_linattn_step(*args)


def ssm_qk_norm_fwd(*args) -> int:
    return _lib().ssm_qk_norm_fwd(*args)


def ssm_qk_norm_bwd(*args) -> int:
    return _lib().ssm_qk_norm_bwd(*args)


def ssm_qk_norm_bwd_workspace_bytes(batch, seqlen, q_heads, k_heads, dim, rot, flags) -> int:
    return _lib().ssm_qk_norm_bwd_workspace_bytes(batch, seqlen, q_heads, k_heads, dim, rot, flags)


# ------------------------------------------------------------------ checks

def _heads_in_place(t):
    """t, or a contiguous copy of a view whose last axis is not contiguous, whose memory holds the
    negative of its values, or whose strides run backwards."""
    t = t.resolve_neg()
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


def _lead_strides(t):
    return (ctypes.c_int64 * (t.dim() - 1))(*t.stride()[:-1])


def _heads(name, t, shape, dtype, dev):
    """An array of heads that the C ABI takes with strides: (tensor, pointer, strides)."""
    _check(name, t, shape, dtype, dev)
    t = _heads_in_place(t)
    return t, t.data_ptr(), _lead_strides(t)


def _decays(g, lead, heads, dev):
    """g as the C ABI takes it: (tensor, pointer, strides); [heads] with strides 0 for the rest."""
    if g is None:
        return None, None, None
    if g.dim() == 1:
        _check("g", g, (heads,), _torch().float32, dev)
    else:
        _check("g", g, (*lead, heads), _torch().float32, dev)
    g = g.resolve_neg()
    strides = (0,) * len(lead) + g.stride() if g.dim() == 1 else g.stride()
    return g, g.data_ptr(), (ctypes.c_int64 * len(strides))(*strides)


def _scale(scale, dk) -> float:
    return max(dk, 1) ** -0.5 if scale is None else float(scale)  # (dk 0 is refused by the library)


class _Sizes:
    """The sizes of a call, from q and v."""

    def __init__(self, q, v):
        if q.dim() != 4 or v.dim() != 4:
            raise ValueError("q and k must be [batch, seqlen, qk_heads, dk] and v [batch, seqlen, "
                             "heads, dv]")
        self.dev, self.flags, self.io = _device("q", q), _io_flag("q", q), q.dtype
        self.batch, self.seqlen, self.qk_heads, self.dk = q.shape
        self.heads, self.dv = v.shape[2:]
        if (self.heads == 0) != (self.qk_heads == 0) or (
                self.qk_heads and self.heads % self.qk_heads):
            raise ValueError("the heads of v must be a multiple of those of q and k")

    @property
    def qk(self):
        return (self.batch, self.seqlen, self.qk_heads, self.dk)

    @property
    def vs(self):
        return (self.batch, self.seqlen, self.heads, self.dv)

    @property
    def state(self):
        return (self.batch, self.heads, self.dv, self.dk)

    @property
    def numbers(self):
        return self.batch, self.seqlen, self.qk_heads, self.heads, self.dk, self.dv


# ------------------------------------------------------------------ linear attention

def linattn(q, k, v, g=None, scale: Optional[float] = None, initial_state=None, lengths=None,
            out=None, final_state=None, return_final_state: bool = True, workspace=None
            ) -> Tuple["torch.Tensor", Optional["torch.Tensor"]]:
    """Linear attention with a decay for each head: S_t = exp(g_t) S_{t-1} + v_t k_t^T and out_t
    = scale S_t q_t.

    q, k: [batch, seqlen, qk_heads, dk], v: [batch, seqlen, heads, dv] (dk and dv at most 256);
    g: log decays, [batch, seqlen, heads] or one for each head [heads], float32 (None: no decay);
    scale: 1 / sqrt(dk) by default; initial_state: [batch, heads, dv, dk] float32 (None: zero);
    lengths: [batch] int32, the steps of each row (clamped to [0, seqlen]; behind them out is 0, the
    state stays and nothing is read). A NaN or infinity is in the results of its own and later steps
    alone (where the recurrence gives an infinity, a result may be NaN). Returns (out [batch,
    seqlen, heads, dv] contiguous in v's dtype, final_state as initial_state). workspace: a uint8
    device tensor of at least ssm_linattn_fwd_workspace_bytes(...) bytes, allocated here when
    None."""
    r = _native().linattn(q, k, v, g, scale, initial_state, lengths, out, final_state,
                          return_final_state, workspace)
    if r is not None:
        return r
    z, f32 = _Sizes(q, v), _torch().float32
    q, qp, qs = _heads("q", q, z.qk, z.io, z.dev)
    k, kp, ks = _heads("k", k, z.qk, z.io, z.dev)
    v, vp, vs = _heads("v", v, z.vs, z.io, z.dev)
    g, gp, gs = _decays(g, (z.batch, z.seqlen), z.heads, z.dev)
    initial_state = _param("initial_state", initial_state, z.state, f32, z.dev)
    lengths = _param("lengths", lengths, (z.batch,), _torch().int32, z.dev)
    if out is None:
        out = v.new_empty(z.vs)
    else:
        _check_out("out", out, z.vs, z.io, z.dev)
    if final_state is not None:
        _check_out("final_state", final_state, z.state, f32, z.dev)
    elif return_final_state:
        final_state = v.new_empty(z.state, dtype=f32)
    workspace = _workspace(workspace, _lib().ssm_linattn_fwd_workspace_bytes(
        z.batch, z.seqlen, z.heads, z.dk, z.dv, z.flags), v)
    _run(_lib().ssm_linattn_fwd, z.dev, qp, qs, kp, ks, vp, vs, gp, gs, _ptr(initial_state),
         _ptr(lengths), _scale(scale, z.dk), z.flags, out.data_ptr(), _ptr(final_state),
         workspace.data_ptr(), workspace.numel(), *z.numbers)
    _wrote(out, final_state)
    return out, final_state


def linattn_backward(q, k, v, dout, g=None, scale: Optional[float] = None, initial_state=None,
                     lengths=None, dfinal=None, want_dg: Optional[bool] = None,
                     want_dinitial: Optional[bool] = None, workspace=None
                     ) -> Dict[str, Optional["torch.Tensor"]]:
    """Gradients of sum(dout * out) + sum(dfinal * final_state) for ``linattn`` on the same
    inputs: dq, dk, dv (contiguous, in the inputs' dtype; dq and dk summed over the heads that
    share them), dg (float32, of g's shape; by default where g is given) and dinitial (float32; by
    default where an initial_state is given), None where not asked for. Bitwise reproducible.
    workspace: a uint8 device tensor of at least ssm_linattn_bwd_workspace_bytes(...) bytes,
    allocated here when None."""
    r = _native().linattn_backward(q, k, v, dout, g, scale, initial_state, lengths, dfinal, want_dg,
                                   want_dinitial, workspace)
    if r is not None:
        return dict(zip(("dq", "dk", "dv", "dg", "dinitial"), r))
    z, f32 = _Sizes(q, v), _torch().float32
    q, qp, qs = _heads("q", q, z.qk, z.io, z.dev)
    k, kp, ks = _heads("k", k, z.qk, z.io, z.dev)
    v, vp, vs = _heads("v", v, z.vs, z.io, z.dev)
    dout, op, os = _heads("dout", dout, z.vs, z.io, z.dev)
    g, gp, gs = _decays(g, (z.batch, z.seqlen), z.heads, z.dev)
    initial_state = _param("initial_state", initial_state, z.state, f32, z.dev)
    dfinal = _param("dfinal", dfinal, z.state, f32, z.dev)
    lengths = _param("lengths", lengths, (z.batch,), _torch().int32, z.dev)
    if want_dg is None:
        want_dg = g is not None
    if want_dg and g is None:
        raise ValueError("want_dg needs g")
    if want_dinitial is None:
        want_dinitial = initial_state is not None
    grads = {"dq": q.new_empty(z.qk), "dk": q.new_empty(z.qk), "dv": q.new_empty(z.vs),
             "dg": q.new_empty(g.shape, dtype=f32) if want_dg else None,
             "dinitial": q.new_empty(z.state, dtype=f32) if want_dinitial else None}
    flags = z.flags | (SSM_LINATTN_HEAD_DG if want_dg and g.dim() == 1 else 0)
    workspace = _workspace(workspace, _lib().ssm_linattn_bwd_workspace_bytes(
        z.batch, z.seqlen, z.heads, z.dk, z.dv, flags), q)
    _run(_lib().ssm_linattn_bwd, z.dev, qp, qs, kp, ks, vp, vs, op, os, gp, gs,
         _ptr(initial_state), _ptr(lengths), _ptr(dfinal), _scale(scale, z.dk), flags,
         grads["dq"].data_ptr(), grads["dk"].data_ptr(), grads["dv"].data_ptr(),
         _ptr(grads["dg"]), _ptr(grads["dinitial"]), workspace.data_ptr(), workspace.numel(),
         *z.numbers)
    return grads


def linattn_step(q, k, v, state, g=None, scale: Optional[float] = None, slots=None, out=None):
    """One token of ``linattn`` for a batch of requests against a cache of states.

    q, k: [batch, qk_heads, dk], v: [batch, heads, dv]; g: [batch, heads] or [heads] float32 (None:
    no decay); state: [nslots, heads, dv, dk] float32 contiguous, updated in place; slots: [batch]
    int32, the slot of each row (None: row i is slot i). A row whose slot lies outside [0,
    nslots) gives 0 and changes nothing; rows naming one slot are successive tokens of it.
    Returns out [batch, heads, dv]."""
    r = _native().linattn_step(q, k, v, state, g, scale, slots, out)
    if r is not None:
        return r
    torch = _torch()
    dev = _device("q", q)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q and k must be [batch, qk_heads, dk], v [batch, heads, dv] and state "
                         "[nslots, heads, dv, dk]")
    flags, io = _io_flag("q", q), q.dtype
    batch, qk_heads, dk = q.shape
    heads, dv = v.shape[1:]
    nslots = state.shape[0]
    if (heads == 0) != (qk_heads == 0) or (qk_heads and heads % qk_heads):
        raise ValueError("the heads of v must be a multiple of those of q and k")
    _check_out("state", state, (nslots, heads, dv, dk), torch.float32, dev)
    q, qp, qs = _heads("q", q, (batch, qk_heads, dk), io, dev)
    k, kp, ks = _heads("k", k, (batch, qk_heads, dk), io, dev)
    v, vp, vs = _heads("v", v, (batch, heads, dv), io, dev)
    g, gp, gs = _decays(g, (batch,), heads, dev)
    slots = _param("slots", slots, (batch,), torch.int32, dev)
    if out is None:
        out = v.new_empty((batch, heads, dv))
    else:
        _check_out("out", out, (batch, heads, dv), io, dev)
    _run(_lib().ssm_linattn_step, dev, qp, qs, kp, ks, vp, vs, gp, gs, _ptr(slots),
         _scale(scale, dk), flags, state.data_ptr(), out.data_ptr(), batch, nslots, qk_heads, heads,
         dk, dv)
    _wrote(state, out)
    return out


# ------------------------------------------------------------------ queries' and keys' norm

def _qk_inputs(q, k, q_weight, k_weight, cos, sin, positions, interleaved):
    torch = _torch()
    dev, f32 = _device("q", q), torch.float32
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [batch, seqlen, heads, dim]")
    flags = _io_flag("q", q) | (SSM_QK_INTERLEAVED if interleaved else 0)
    batch, seqlen, q_heads, dim = q.shape
    k_heads = k.shape[2]
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    rot = rows = 0
    if cos is not None:
        if cos.dim() != 2 or 2 * cos.shape[1] > dim:
            raise ValueError("cos and sin must be [positions, at most dim / 2]")
        rows, rot = cos.shape[0], 2 * cos.shape[1]
        cos = _param("cos", cos, (rows, rot // 2), f32, dev)
        sin = _param("sin", sin, (rows, rot // 2), f32, dev)
        if positions is None and rows < seqlen:
            raise ValueError(f"cos and sin have {rows} positions for {seqlen} steps")
    q, qp, qs = _heads("q", q, (batch, seqlen, q_heads, dim), q.dtype, dev)
    k, kp, ks = _heads("k", k, (batch, seqlen, k_heads, dim), q.dtype, dev)
    shared = (_param("q_weight", q_weight, (dim,), f32, dev),
              _param("k_weight", k_weight, (dim,), f32, dev), cos, sin,
              _param("positions", positions, (batch, seqlen), torch.int32, dev))
    return (dev, flags, (q, k), (qp, qs, kp, ks), shared,
            (batch, seqlen, q_heads, k_heads, dim, rot, rows))


def qk_norm(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
            eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None
            ) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """RMS norm of each head's queries and keys, and the position rotation of the first
    2 cos.shape[1] values of each head, in one pass.

    q: [batch, seqlen, q_heads, dim], k: [batch, seqlen, k_heads, dim] float32 or bfloat16 (dim at
    most 256); q_weight, k_weight: [dim] float32 (None: ones); cos, sin: [positions, pairs]
    float32, the angles' (None: no rotation); positions: [batch, seqlen] int32 (None: step t is
    at position t); a step whose position lies outside the table, or without one below 0, is padding
    and gives zeros. Pairs are (i, i + pairs), or, interleaved, (2 i, 2 i + 1). Returns (q_out,
    k_out), contiguous, in q's dtype."""
    r = _native().qk_norm(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out,
                          k_out)
    if r is not None:
        return r
    dev, flags, (q, k), pointers, shared, sizes = _qk_inputs(q, k, q_weight, k_weight, cos, sin,
                                                             positions, interleaved)
    if q_out is None:
        q_out = q.new_empty(q.shape)
    else:
        _check_out("q_out", q_out, q.shape, q.dtype, dev)
    if k_out is None:
        k_out = k.new_empty(k.shape)
    else:
        _check_out("k_out", k_out, k.shape, q.dtype, dev)
    _run(_lib().ssm_qk_norm_fwd, dev, *pointers, *map(_ptr, shared), eps, flags, q_out.data_ptr(),
         k_out.data_ptr(), *sizes)
    _wrote(q_out, k_out)
    return q_out, k_out


def qk_norm_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None,
                     positions=None, eps: float = 1e-6, interleaved: bool = False, workspace=None
                     ) -> Dict[str, Optional["torch.Tensor"]]:
    """Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) for ``qk_norm`` on the same inputs:
    dq and dk (contiguous, in q's dtype), dq_weight and dk_weight (float32; None without the
    weight). Bitwise reproducible. workspace: a uint8 device tensor of at least
    ssm_qk_norm_bwd_workspace_bytes(...) bytes, allocated here when None."""
    r = _native().qk_norm_backward(q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions, eps,
                                   interleaved, workspace)
    if r is not None:
        return dict(zip(("dq", "dk", "dq_weight", "dk_weight"), r))
    f32 = _torch().float32
    dev, flags, (q, k), pointers, shared, sizes = _qk_inputs(q, k, q_weight, k_weight, cos, sin,
                                                             positions, interleaved)
    dq_out, dqp, dqs = _heads("dq_out", dq_out, q.shape, q.dtype, dev)
    dk_out, dkp, dks = _heads("dk_out", dk_out, k.shape, q.dtype, dev)
    dim = sizes[4]
    grads = {"dq": q.new_empty(q.shape), "dk": k.new_empty(k.shape),
             "dq_weight": None if q_weight is None else q.new_empty((dim,), dtype=f32),
             "dk_weight": None if k_weight is None else q.new_empty((dim,), dtype=f32)}
    workspace = _workspace(
        workspace, _lib().ssm_qk_norm_bwd_workspace_bytes(*sizes[:6], flags), q)
    _run(_lib().ssm_qk_norm_bwd, dev, *pointers, dqp, dqs, dkp, dks, *map(_ptr, shared), eps, flags,
         *(_ptr(t) for t in grads.values()), workspace.data_ptr(), workspace.numel(), *sizes)
    return grads


# ------------------------------------------------------------------ autograd

_functions = None


def _autograd():
    """The torch.autograd.Functions behind ``linear_attention`` and ``rotary_qk_norm`` (built on
    first use, so that importing this module does not import torch)."""
    global _functions
    if _functions is not None:
        return _functions
    import torch
    from torch.autograd.function import once_differentiable

    class LinearAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g, scale, initial_state, lengths):
            out, fin = linattn(q, k, v, g, scale=scale, initial_state=initial_state,
                               lengths=lengths)
            ctx.save_for_backward(q, k, v, g, initial_state, lengths)
            ctx.scale = scale
            ctx.set_materialize_grads(False)
            return out, fin

        @staticmethod
        @once_differentiable
        def backward(ctx, dout, dfin):
            q, k, v, g, initial_state, lengths = ctx.saved_tensors
            dout = v.new_zeros(v.shape) if dout is None else dout
            d = linattn_backward(q, k, v, dout, g, scale=ctx.scale, initial_state=initial_state,
                                 lengths=lengths, dfinal=dfin,
                                 want_dg=g is not None and ctx.needs_input_grad[3],
                                 want_dinitial=ctx.needs_input_grad[5])
            return d["dq"], d["dk"], d["dv"], d["dg"], None, d["dinitial"], None

    class RotaryQkNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
            outs = qk_norm(q, k, q_weight, k_weight, cos, sin, positions=positions, eps=eps,
                           interleaved=interleaved)
            ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
            ctx.options = dict(eps=eps, interleaved=interleaved)
            return outs

        @staticmethod
        @once_differentiable
        def backward(ctx, dq_out, dk_out):
            q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
            d = qk_norm_backward(q, k, dq_out, dk_out, q_weight, k_weight, cos, sin,
                                 positions=positions, **ctx.options)
            return (d["dq"], d["dk"], d["dq_weight"], d["dk_weight"], None, None, None, None,
                    None)

    _functions = (LinearAttention, RotaryQkNorm)
    return _functions


def linear_attention(q, k, v, g=None, scale: Optional[float] = None, initial_state=None,
                     lengths=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """Differentiable ``linattn``: (out, final_state), with gradients for q, k, v, g and
    initial_state through autograd (``linattn_backward``)."""
    return _autograd()[0].apply(q, k, v, g, scale, initial_state, lengths)


def rotary_qk_norm(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                   eps: float = 1e-6, interleaved: bool = False
                   ) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """Differentiable ``qk_norm``, with gradients for q, k and the weights through autograd
    (``qk_norm_backward``); the angles are constants."""
    for name, t in (("cos", cos), ("sin", sin)):
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} has no gradient here")
    return _autograd()[1].apply(q, k, q_weight, k_weight, cos, sin, positions, float(eps),
                                bool(interleaved))
