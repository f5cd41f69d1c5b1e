"""Pins of the oracles of linear attention and of the queries' and keys' norm (oracle/linattn.py), on
the CPU: gradients against central differences (as in test_oracle_block_pins.py, bar 1e-6), the
recurrence against its unrolled sums, the step against the prompt, the rotation's invariants."""
import numpy as np
import pytest

from oracle import block as ob
from oracle import linattn as ol
from test_oracle_block_pins import near, numeric


def make(seed, b=2, L=5, hk=2, h=4, dk=3, dv=2):
    r = np.random.default_rng(seed)
    mk = lambda *s: r.standard_normal(s)
    return dict(q=mk(b, L, hk, dk), k=mk(b, L, hk, dk), v=mk(b, L, h, dv), g=-np.abs(mk(b, L, h)),
                s0=mk(b, h, dv, dk), dout=mk(b, L, h, dv), ds=mk(b, h, dv, dk))


@pytest.mark.parametrize("lengths", [None, [5, 2], [0, 4]])
def test_linattn_gradients(lengths):
    x = make(3)

    def loss():
        o, s = ol.linattn_ref(x["q"], x["k"], x["v"], x["g"], 0.7, x["s0"], lengths)
        return (o * x["dout"]).sum() + (s * x["ds"]).sum()

    d = ol.linattn_bwd_ref(x["q"], x["k"], x["v"], x["dout"], x["g"], 0.7, x["s0"], lengths, x["ds"])
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dinitial", "s0")):
        near(d[name], numeric(loss, x[key]), 1e-6)


def test_linattn_head_decay_gradient():
    x = make(4)
    g = -np.abs(np.random.default_rng(5).standard_normal(4))
    loss = lambda: (ol.linattn_ref(x["q"], x["k"], x["v"], g)[0] * x["dout"]).sum()
    d = ol.linattn_bwd_ref(x["q"], x["k"], x["v"], x["dout"], g)
    near(d["dg"].sum((0, 1)), numeric(loss, g), 1e-6)


def test_linattn_unrolled():
    """out_t = scale sum_s exp(sum of g in (s, t]) (q_t . k_s) v_s + the state's part."""
    x = make(6)
    out, fin = ol.linattn_ref(x["q"], x["k"], x["v"], x["g"], 0.5, x["s0"])
    cs = np.cumsum(x["g"], 1)
    want = np.zeros_like(out)
    for b, t, h in np.ndindex(2, 5, 4):
        for s in range(t + 1):
            w = np.exp(cs[b, t, h] - cs[b, s, h]) * (x["q"][b, t, h // 2] @ x["k"][b, s, h // 2])
            want[b, t, h] += 0.5 * w * x["v"][b, s, h]
        want[b, t, h] += 0.5 * np.exp(cs[b, t, h]) * (x["s0"][b, h] @ x["q"][b, t, h // 2])
    near(out, want, 1e-12)


def test_linattn_step_is_the_prompt():
    x = make(7)
    out, fin = ol.linattn_ref(x["q"], x["k"], x["v"], x["g"], None, x["s0"])
    cache = x["s0"].copy()
    for t in range(5):
        o, cache = ol.linattn_step_ref(x["q"][:, t], x["k"][:, t], x["v"][:, t], cache, x["g"][:, t])
        near(o, out[:, t], 1e-12)
    near(cache, fin, 1e-12)


def test_ssd_is_linattn_with_one_key():
    """Mamba-2's step is linear attention with B as the key, C as the query, dt x as the value and
    dt A as the log decay."""
    r = np.random.default_rng(8)
    b, heads, p, n = 2, 3, 2, 4
    x, dt = r.standard_normal((b, heads * p)), np.abs(r.standard_normal((b, heads)))
    A, B, C = -np.abs(r.standard_normal(heads)), r.standard_normal((b, n)), r.standard_normal((b, n))
    state = r.standard_normal((b, heads * p, n))
    want, after = ob.step_ref(x, dt, A, B, C, state, None, None, None, False, None)
    v = x.reshape(b, heads, p) * dt[:, :, None]
    out, cache = ol.linattn_step_ref(C[:, None], B[:, None], v, state.reshape(b, heads, p, n),
                                     dt * A, scale=1.0)
    near(out.reshape(b, -1), want, 1e-12)
    near(cache.reshape(after.shape), after, 1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 2, 6])
def test_qk_norm_gradients(rot, interleaved):
    r = np.random.default_rng(rot)
    x, w, dout = r.standard_normal((2, 3, 2, 6)), r.standard_normal(6), r.standard_normal((2, 3, 2, 6))
    angle = r.standard_normal((5, rot // 2))
    cos, sin = (np.cos(angle), np.sin(angle)) if rot else (None, None)
    pos = np.array([[0, 4, -1], [5, 2, 2]]) if rot else None
    opt = dict(cos=cos, sin=sin, positions=pos, eps=0.1, interleaved=interleaved)
    loss = lambda: (ol.qk_norm_ref(x, w, **opt) * dout).sum()
    dx, dw = ol.qk_norm_bwd_ref(x, dout, w, **opt)
    near(dx, numeric(loss, x), 1e-6)
    near(dw, numeric(loss, w), 1e-6)


def test_qk_norm_rotation():
    """A rotation keeps each pair's length; two steps' product depends on the angles' difference."""
    r = np.random.default_rng(9)
    x, y = r.standard_normal((1, 4, 1, 8)), r.standard_normal((1, 4, 1, 8))
    angle = np.arange(10)[:, None] * np.array([1.0, 0.1, 0.01, 0.001])
    cos, sin = np.cos(angle), np.sin(angle)
    for inter in (False, True):
        turn = lambda v, shift: ol.qk_norm_ref(v, None, cos, sin, np.arange(4)[None] + shift,
                                               interleaved=inter)
        flat = ol.qk_norm_ref(x, None)
        near((turn(x, 0) ** 2).sum(-1), (flat ** 2).sum(-1), 1e-12)
        near((turn(x, 0) * turn(y, 0)).sum(-1), (turn(x, 5) * turn(y, 5)).sum(-1), 1e-12)
