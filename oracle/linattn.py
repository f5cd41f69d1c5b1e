"""Oracles of linear attention with a decay for each head and of the queries' and keys' norm, float64
(TEST INFRASTRUCTURE ONLY): the recurrence step by step, its adjoint step by step from the last,
and each head's norm and rotation. Nothing is shared with the GPU library.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np

from .block import _ends, _f64


def _gates(g, batch, seqlen, heads):
    """[batch, seqlen, heads] decay factors."""
    if g is None:
        return np.ones((batch, seqlen, heads))
    with np.errstate(over="ignore"):
        return np.exp(np.broadcast_to(_f64(g), (batch, seqlen, heads)))


def linattn_ref(q, k, v, g=None, scale=None, initial_state=None, lengths=None
                ) -> Tuple[np.ndarray, np.ndarray]:
    """(out, final_state): S = exp(g) S + v k^T, out = scale S q, one step at a time."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    batch, seqlen, heads, dv = v.shape
    dk, group = q.shape[3], heads // q.shape[2]
    scale = dk ** -0.5 if scale is None else scale
    a = _gates(g, batch, seqlen, heads)
    out = np.zeros(v.shape)
    final = np.zeros((batch, heads, dv, dk))
    for b, n in enumerate(_ends(lengths, batch, seqlen)):
        S = np.zeros((heads, dv, dk)) if initial_state is None else _f64(initial_state)[b].copy()
        for t in range(n):
            kt, qt = np.repeat(k[b, t], group, 0), np.repeat(q[b, t], group, 0)
            S = a[b, t][:, None, None] * S + v[b, t][:, :, None] * kt[:, None]
            out[b, t] = scale * (S * qt[:, None]).sum(2)
        final[b] = S
    return out, final


def linattn_bwd_ref(q, k, v, dout, g=None, scale=None, initial_state=None, lengths=None,
                    dfinal=None) -> Dict[str, np.ndarray]:
    """Gradients of sum(dout out) + sum(dfinal final_state): every state kept, then the adjoint R of
    the state from the last step on. dg has [batch, seqlen, heads] entries, whatever g's shape."""
    q, k, v, dout = _f64(q), _f64(k), _f64(v), _f64(dout)
    batch, seqlen, heads, dv = v.shape
    qk_heads, dk = q.shape[2:]
    group = heads // qk_heads
    scale = dk ** -0.5 if scale is None else scale
    a = _gates(g, batch, seqlen, heads)
    d = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape),
         "dg": np.zeros((batch, seqlen, heads)), "dinitial": np.zeros((batch, heads, dv, dk))}
    shared = lambda x: x.reshape(qk_heads, group, dk).sum(1)
    for b, n in enumerate(_ends(lengths, batch, seqlen)):
        S = [np.zeros((heads, dv, dk)) if initial_state is None else _f64(initial_state)[b]]
        for t in range(n):
            S.append(a[b, t][:, None, None] * S[-1]
                     + v[b, t][:, :, None] * np.repeat(k[b, t], group, 0)[:, None])
        R = np.zeros((heads, dv, dk)) if dfinal is None else _f64(dfinal)[b].copy()
        for t in range(n - 1, -1, -1):
            kt, qt = np.repeat(k[b, t], group, 0), np.repeat(q[b, t], group, 0)
            R = R + scale * dout[b, t][:, :, None] * qt[:, None]
            d["dq"][b, t] = shared(scale * (S[t + 1] * dout[b, t][:, :, None]).sum(1))
            d["dk"][b, t] = shared((R * v[b, t][:, :, None]).sum(1))
            d["dv"][b, t] = (R * kt[:, None]).sum(2)
            d["dg"][b, t] = a[b, t] * (R * S[t]).sum((1, 2))
            R = a[b, t][:, None, None] * R
        d["dinitial"][b] = R
    return d


def linattn_step_ref(q, k, v, state, g=None, scale=None, slots=None
                     ) -> Tuple[np.ndarray, np.ndarray]:
    """(out, the cache afterwards): one token a row, in row order."""
    q, k, v, state = _f64(q), _f64(k), _f64(v), _f64(state).copy()
    batch, heads, _ = v.shape
    dk, group = q.shape[2], heads // q.shape[1]
    scale = dk ** -0.5 if scale is None else scale
    a = _gates(g, batch, 1, heads)[:, 0] if g is None or np.ndim(g) == 1 else np.exp(_f64(g))
    out = np.zeros(v.shape)
    for i in range(batch):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < state.shape[0]:
            continue
        kt, qt = np.repeat(k[i], group, 0), np.repeat(q[i], group, 0)
        state[s] = a[i][:, None, None] * state[s] + v[i][:, :, None] * kt[:, None]
        out[i] = scale * (state[s] * qt[:, None]).sum(2)
    return out, state


def _turn(x, cos, sin, rot, interleaved):
    y = x.copy()
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + (1 if interleaved else rot // 2)
    y[..., i], y[..., j] = x[..., i] * cos - x[..., j] * sin, x[..., j] * cos + x[..., i] * sin
    return y


def _angles(cos, sin, positions, batch, seqlen):
    """(cos, sin [batch, seqlen, 1, pairs], whether each step has a position)."""
    if cos is None:
        return np.ones((1, 1, 1, 0)), np.zeros((1, 1, 1, 0)), np.ones((batch, seqlen), bool), 0
    at = np.broadcast_to(np.arange(seqlen), (batch, seqlen)) if positions is None else positions
    on = (at >= 0) & (at < len(cos))
    at = np.where(on, at, 0)
    if len(cos) == 0:
        cos = sin = np.zeros((1, cos.shape[1]))
    return _f64(cos)[at][:, :, None], _f64(sin)[at][:, :, None], on, 2 * cos.shape[1]


def qk_norm_ref(x, weight=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """One side (queries or keys): [batch, seqlen, heads, dim]."""
    x = _f64(x)
    c, s, on, rot = _angles(cos, sin, positions, *x.shape[:2])
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = y if weight is None else y * _f64(weight)
    return np.where(on[:, :, None, None], _turn(y, c, s, rot, interleaved), 0.0)


def qk_norm_bwd_ref(x, dout, weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                    interleaved=False) -> Tuple[np.ndarray, np.ndarray]:
    """(dx, dweight) of one side."""
    x, dout = _f64(x), _f64(dout)
    c, s, on, rot = _angles(cos, sin, positions, *x.shape[:2])
    dy = np.where(on[:, :, None, None], _turn(dout, c, -s, rot, interleaved), 0.0)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    u = dy if weight is None else dy * _f64(weight)
    return r * (u - n * (u * n).mean(-1, keepdims=True)), (dy * n).sum((0, 1, 2))
