"""Pins of the oracles of the operators around the scan (oracle/block.py), on the CPU.

Gradients against central differences of the forward: with a step h the difference is off by
h^2/6 times a third derivative plus eps/h of the loss; at h = 1e-5 and values of order one that
is below 1e-8 relative to the largest gradient, and the bar is 1e-6. The steps against the
whole-prompt oracles: the same sums in float64, 1e-12.
"""
import numpy as np
import pytest

import oracle
from oracle import block as ob


def numeric(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


def near(got, want, tol):
    scale = max(np.abs(want).max(), 1e-30)
    assert np.abs(got - want).max() <= tol * scale, np.abs(got - want).max() / scale


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_gradients(width, silu):
    r = np.random.default_rng(width)
    b, d, L = 3, 2, 6
    x, w, bias = r.standard_normal((b, d, L)), r.standard_normal((d, width)), r.standard_normal(d)
    init = r.standard_normal((b, d, width - 1))
    dout, dfin = r.standard_normal((b, d, L)), r.standard_normal((b, d, width - 1))
    lengths = [6, 1, 0]

    def loss():
        out, fin = ob.conv_ref(x, w, bias, silu, init, lengths)
        return (out * dout).sum() + (fin * dfin).sum()

    g = ob.conv_bwd_ref(x, w, dout, bias, silu, init, lengths, dfin)
    for name, v in (("dx", x), ("dweight", w), ("dbias", bias), ("dinitial", init)):
        near(g[name], numeric(loss, v), 1e-6)


def test_conv_is_a_correlation_and_hands_its_state_on():
    r = np.random.default_rng(7)
    x, w = r.standard_normal((1, 3, 20)), r.standard_normal((3, 4))
    out, fin = ob.conv_ref(x, w)
    for d in range(3):
        assert np.allclose(out[0, d], np.convolve(x[0, d], w[d, ::-1])[:20], rtol=0, atol=1e-12)
    assert np.array_equal(fin[0], x[0, :, -3:])
    o1, f1 = ob.conv_ref(x[..., :2], w)
    o2, f2 = ob.conv_ref(x[..., 2:], w, initial_state=f1)
    near(np.concatenate((o1, o2), 2), out, 1e-12)
    assert np.array_equal(f2, fin)


def test_conv_steps_equal_the_prompt():
    r = np.random.default_rng(8)
    x, w, bias = r.standard_normal((2, 3, 5)), r.standard_normal((3, 3)), r.standard_normal(3)
    state = np.zeros((4, 3, 2))
    outs = []
    for t in range(5):
        o, state = ob.conv_step_ref(x[..., t], state, w, bias, True, slots=[3, 1])
        outs.append(o)
    out, fin = ob.conv_ref(x, w, bias, True)
    near(np.stack(outs, 2), out, 1e-12)
    assert np.array_equal(state[[3, 1]], fin) and not state[[0, 2]].any()


@pytest.mark.parametrize("heads", [None, 2])
def test_state_steps_equal_the_scan(heads):
    r = np.random.default_rng(9)
    b, d, n, L = 2, 6, 5, 4
    x, z = r.standard_normal((b, d, L)), r.standard_normal((b, d, L))
    B, C = r.standard_normal((b, n, L)), r.standard_normal((b, n, L))
    steps = d if heads is None else heads
    dt, bias, D = r.standard_normal((b, steps, L)), r.standard_normal(steps), r.standard_normal(d)
    A = -np.exp(r.standard_normal((d, n) if heads is None else heads))
    state = r.standard_normal((3, d, n))
    h0 = state[[2, 0]].copy()
    outs = []
    for t in range(L):
        o, state = ob.step_ref(x[..., t], dt[..., t], A, B[..., t], C[..., t], state, D,
                               z[..., t], bias, True, slots=[2, 0])
        outs.append(o)
    ref = oracle.scan_ref if heads is None else oracle.ssd_ref
    out, fin = ref(x, dt, A, B, C, D, z, bias, True, h0)
    near(np.stack(outs, 2), out, 1e-12)
    near(state[[2, 0]], fin, 1e-12)


def test_rows_of_one_slot_are_successive_tokens():
    r = np.random.default_rng(10)
    x, w = r.standard_normal((3, 2)), r.standard_normal((2, 2))
    out, state = ob.conv_step_ref(x, np.zeros((1, 2, 1)), w, slots=[0, -1, 0])
    whole, fin = ob.conv_ref(x[[0, 2]].T[None], w)
    near(out[[0, 2]].T[None], whole, 1e-12)
    assert not out[1].any() and np.array_equal(state, fin)


@pytest.mark.parametrize("gate", ["none", "first", "last"])
@pytest.mark.parametrize("groups", [1, 3])
def test_norm_gradients(groups, gate):
    r = np.random.default_rng(11 + groups)
    b, d, L = 2, 6, 3
    y, w, dout = r.standard_normal((b, d, L)), r.standard_normal(d), r.standard_normal((b, d, L))
    z = None if gate == "none" else r.standard_normal((b, d, L))
    last = gate == "last"

    def loss():
        return (ob.norm_ref(y, w, z, 1e-5, groups, last)[0] * dout).sum()

    g = ob.norm_bwd_ref(y, w, dout, z, 1e-5, groups, last)
    near(g["dy"], numeric(loss, y), 1e-6)
    near(g["dweight"], numeric(loss, w), 1e-6)
    if z is None:
        assert g["dz"] is None
    else:
        near(g["dz"], numeric(loss, z), 1e-6)


def test_norm_values():
    y = np.array([[[3.0], [4.0], [0.0], [5.0]]])
    out, rstd = ob.norm_ref(y, np.ones(4), eps=0.0, groups=2)
    assert np.allclose(rstd[0, :, 0], [1 / np.sqrt(12.5)] * 2)
    assert np.allclose(out[0, :, 0], y[0, :, 0] / np.sqrt(12.5))
