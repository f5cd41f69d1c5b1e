"""Oracles of the operators around the scan, float64 (TEST INFRASTRUCTURE ONLY): the short causal
convolution, the single-token state steps, the gated RMS norm, and the gradients of the first
and the last. Each is written from its definition, one token or tap at a time where that is
the definition, and shares nothing with the GPU library.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(x):
    return np.logaddexp(0.0, x)


def _ends(lengths, batch, seqlen):
    if lengths is None:
        return [seqlen] * batch
    return [min(max(int(n), 0), seqlen) for n in lengths]


def conv_ref(x, weight, bias=None, silu=False, initial_state=None, lengths=None
             ) -> Tuple[np.ndarray, np.ndarray]:
    """(out, final_state): a shift register of width - 1 inputs per channel, one step at a time."""
    x, weight, bias = _f64(x), _f64(weight), _f64(bias)
    batch, dim, seqlen = x.shape
    width = weight.shape[1]
    out = np.zeros_like(x)
    final = np.zeros((batch, dim, width - 1))
    for b, n in enumerate(_ends(lengths, batch, seqlen)):
        past = np.zeros((dim, width - 1)) if initial_state is None else _f64(initial_state)[b].copy()
        for t in range(n):
            window = np.concatenate((past, x[b, :, t:t + 1]), axis=1)
            p = (window * weight).sum(1) + (0.0 if bias is None else bias)
            out[b, :, t] = p * sigmoid(p) if silu else p
            past = window[:, 1:]
        final[b] = past
    return out, final


def conv_bwd_ref(x, weight, dout, bias=None, silu=False, initial_state=None, lengths=None,
                 dfinal=None) -> Dict[str, np.ndarray]:
    """Gradients of sum(dout out) + sum(dfinal final_state), step by step from the last."""
    x, weight, bias, dout = _f64(x), _f64(weight), _f64(bias), _f64(dout)
    batch, dim, seqlen = x.shape
    width = weight.shape[1]
    dx = np.zeros_like(x)
    dw, db = np.zeros((dim, width)), np.zeros(dim)
    dinit = np.zeros((batch, dim, width - 1))
    for b, n in enumerate(_ends(lengths, batch, seqlen)):
        first = np.zeros((dim, width - 1)) if initial_state is None else _f64(initial_state)[b]
        e = np.concatenate((first, x[b, :, :n]), axis=1)
        de = np.zeros_like(e)
        if dfinal is not None:
            de[:, n:] += _f64(dfinal)[b]
        for t in range(n):
            window = e[:, t:t + width]
            p = (window * weight).sum(1) + (0.0 if bias is None else bias)
            s = sigmoid(p)
            dp = dout[b, :, t] * (s * (1 + p * (1 - s)) if silu else 1.0)
            dw += dp[:, None] * window
            db += dp
            de[:, t:t + width] += dp[:, None] * weight
        dinit[b] = de[:, :width - 1]
        dx[b, :, :n] = de[:, width - 1:]
    return {"dx": dx, "dweight": dw, "dbias": db, "dinitial": dinit}


def conv_step_ref(x, state, weight, bias=None, silu=False, slots=None):
    """(out, state after): rows one after the other."""
    x, state, weight, bias = _f64(x), _f64(state).copy(), _f64(weight), _f64(bias)
    out = np.zeros_like(x)
    for i in range(x.shape[0]):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < state.shape[0]:
            continue
        window = np.concatenate((state[s], x[i][:, None]), axis=1)
        p = (window * weight).sum(1) + (0.0 if bias is None else bias)
        out[i] = p * sigmoid(p) if silu else p
        state[s] = window[:, 1:]
    return out, state


def step_ref(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=False, slots=None):
    """(out, state after) of scan_step (A [dim, dstate]) or ssd_step (A [nheads]), rows one
    after the other."""
    x, dt, A, B, C, D, z, dt_bias = (_f64(v) for v in (x, dt, A, B, C, D, z, dt_bias))
    state = _f64(state).copy()
    out = np.zeros_like(x)
    dim = x.shape[1]
    per = 1 if A.ndim == 2 else dim // A.shape[0]
    for i in range(x.shape[0]):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < state.shape[0]:
            continue
        step = dt[i] + (0.0 if dt_bias is None else dt_bias)
        if dt_softplus:
            step = softplus(step)
        step = np.repeat(step, per)
        a = A if A.ndim == 2 else np.repeat(A, per)[:, None]
        h = np.exp(step[:, None] * a) * state[s] + (step * x[i])[:, None] * B[i][None, :]
        y = h @ C[i]
        if D is not None:
            y = y + D * x[i]
        if z is not None:
            y = y * z[i] * sigmoid(z[i])
        out[i], state[s] = y, h
    return out, state


def _norm_parts(y, z, eps, groups, norm_before_gate):
    b, d, L = y.shape
    gate = np.ones_like(y) if z is None else z * sigmoid(z)
    v = y if norm_before_gate else y * gate
    mean = (v.reshape(b, groups, d // groups, L) ** 2).mean(2)
    rstd = 1.0 / np.sqrt(mean + eps)
    return gate, v, rstd, np.repeat(rstd, d // groups, axis=1)


def norm_ref(y, weight, z=None, eps=1e-5, groups=1, norm_before_gate=False):
    """(out [batch, dim, seqlen], rstd [batch, groups, seqlen])."""
    y, weight, z = _f64(y), _f64(weight), _f64(z)
    gate, v, rstd, r = _norm_parts(y, z, eps, groups, norm_before_gate)
    out = v * r * weight[None, :, None]
    return (out * gate if norm_before_gate else out), rstd


def norm_bwd_ref(y, weight, dout, z=None, eps=1e-5, groups=1, norm_before_gate=False
                 ) -> Dict[str, Optional[np.ndarray]]:
    """Gradients of sum(dout out), through the normed values n = v r: dv = r (dn - n mean(dn n))."""
    y, weight, z, g = _f64(y), _f64(weight), _f64(z), _f64(dout)
    b, d, L = y.shape
    gate, v, _, r = _norm_parts(y, z, eps, groups, norm_before_gate)
    n = v * r
    dgate = None
    if z is not None:
        s = sigmoid(z)
        dgate = s * (1 + z * (1 - s))
    into = g * gate if norm_before_gate else g
    dn = into * weight[None, :, None]
    m = (dn * n).reshape(b, groups, d // groups, L).mean(2)
    dv = r * (dn - n * np.repeat(m, d // groups, axis=1))
    out = {"dweight": (into * n).sum((0, 2)), "dy": dv if norm_before_gate else dv * gate,
           "dz": None}
    if z is not None:
        out["dz"] = (g * weight[None, :, None] * n if norm_before_gate else dv * y) * dgate
    return out
