"""GPU parity of linear attention with a decay for each head (linattn, its gradient, linattn_step)
against the float64 oracle (oracle/linattn.py, pinned in test_oracle_linattn_pins.py), element by
element within the bounds of linattn_util.py.

Cover: one step to many chunks and segments, head sizes from 1 to 256, shared queries and keys,
both storage types, every form of decay, ragged rows with NaN behind them, strided inputs, states
in and out, extreme decays, caches past 2^31 states, repeated and missing slots.
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import Rand, same
from gpu_util import announce, host, torch
from linattn_util import Attention, reach, roundings, within
from oracle import linattn as ol

pytestmark = pytest.mark.gpu

# batch, steps, query heads, heads, dk, dv, decay, lengths, state
SHAPES = [
    (1, 1, 1, 1, 16, 16, "token", None, True),
    (2, 3, 1, 2, 1, 1, "head", None, True),
    (1, 64, 1, 1, 64, 64, "none", None, False),
    (2, 65, 2, 2, 33, 17, "token", [65, 1], True),
    (1, 130, 1, 4, 128, 64, "token", None, False),
    (3, 200, 2, 2, 96, 80, "token", [200, 0, 131], True),
    (1, 70, 1, 1, 256, 256, "head", None, True),
    (1, 600, 1, 1, 20, 130, "head", None, True),
    (2, 97, 3, 6, 64, 128, "none", [-3, 500], True),
    (1, 129, 1, 2, 200, 48, "token", [128], False),
]
IDS = ["b{}L{}hk{}h{}k{}v{}{}".format(*s[:7]) for s in SHAPES]


def make(shape, io, **kw):
    b, L, hk, h, dk, dv, decay, lengths, state = shape
    return Attention(b, L, hk, h, dk, dv, io, decay, lengths, state, **kw)


def check_forward(a, out, fin, label):
    ref, rfin = ol.linattn_ref(a.q64, a.k64, a.v64, **a.ref_args())
    ab, afin = ol.linattn_ref(*map(np.abs, (a.q64, a.k64, a.v64)), **a.abs_args())
    within(out, ref, ab, a.io, a.roundings, label + " out")
    within(fin, rfin, afin, "f32", a.roundings, label + " final")


def check_backward(a, d, label):
    ref = ol.linattn_bwd_ref(a.q64, a.k64, a.v64, a.dout64, dfinal=a.ds64, **a.ref_args())
    ab = ol.linattn_bwd_ref(*map(np.abs, (a.q64, a.k64, a.v64, a.dout64)),
                            dfinal=None if a.ds64 is None else np.abs(a.ds64), **a.abs_args())
    for name in ("dq", "dk", "dv"):
        within(d[name], ref[name], ab[name], a.io, a.roundings, f"{label} {name}")
    if a.s0 is not None:
        within(d["dinitial"], ref["dinitial"], ab["dinitial"], "f32", a.roundings, label + " dinitial")
    if a.g is not None:
        far = reach(ab["dg"])
        got, want = d["dg"], ref["dg"]
        if a.g.dim() == 1:
            want, far = want.sum((0, 1)), far.sum((0, 1))
        within(got, want, far, "f32", 2 * a.roundings, label + " dg")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, io):
    announce(f"linattn {shape} {io}")
    a = make(shape, io, seed=11)
    out, fin = ssm.linattn(a.q, a.k, a.v, **a.args())
    check_forward(a, out, fin, "linattn")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape, io):
    announce(f"linattn_backward {shape} {io}")
    a = make(shape, io, seed=12)
    d = ssm.linattn_backward(a.q, a.k, a.v, a.dout, dfinal=a.ds, **a.args())
    assert (d["dg"] is None) == (a.g is None) and (d["dinitial"] is None) == (a.s0 is None)
    check_backward(a, d, "gradient")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 2, 8])
def test_strides(offset, io):
    """Slices at odd places, head-major views and broadcast rows give the bits of contiguous inputs."""
    t = torch()
    announce(f"linattn strides offset {offset} {io}")
    a = make((2, 100, 2, 4, 40, 24, "token", None, True), io, seed=13, offset=offset)
    opt = a.args()
    want = ssm.linattn(*(x.contiguous() for x in (a.q, a.k, a.v)), **opt)
    grads = ssm.linattn_backward(*(x.contiguous() for x in (a.q, a.k, a.v)), a.dout, dfinal=a.ds, **opt)
    major = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)
    for form in (lambda x: x, major):
        got = ssm.linattn(form(a.q), form(a.k), form(a.v), g=major(a.g),
                          initial_state=a.s0, lengths=a.n)
        assert all(same(x, y) for x, y in zip(got, want))
        d = ssm.linattn_backward(form(a.q), form(a.k), form(a.v), form(a.dout), dfinal=a.ds, **opt)
        assert all(same(d[n], grads[n]) for n in grads)
    one = lambda x: x[:1].expand(2, *x.shape[1:])
    got = ssm.linattn(one(a.q), one(a.k), one(a.v), g=one(a.g))
    want = ssm.linattn(a.q[:1], a.k[:1], a.v[:1], g=a.g[:1])
    assert same(got[0][1], want[0][0]) and same(got[1][0], want[1][0])
    last = a.q.transpose(2, 3).contiguous().transpose(2, 3)  # not contiguous in dk: copied
    assert same(ssm.linattn(last, a.k, a.v, **opt)[0], ssm.linattn(a.q, a.k, a.v, **opt)[0])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_extreme_decays(io):
    """Resets (-inf), decays far below what a float's exponential holds, growth, no decay at all."""
    t = torch()
    announce(f"linattn extreme decays {io}")
    a = make((1, 150, 1, 6, 32, 32, "token", None, True), io, seed=14)
    a.g[:, ::7, 0] = float("-inf")
    a.g[..., 1] = -90.0
    a.g[..., 2] = float("-inf")
    a.g[..., 3] = 0.02
    a.g[..., 4] = 0.0
    a.g[:, 75:, 5] = -3e38
    a.g64 = host(a.g)
    out, fin = ssm.linattn(a.q, a.k, a.v, **a.args())
    check_forward(a, out, fin, "extreme")
    check_backward(a, ssm.linattn_backward(a.q, a.k, a.v, a.dout, dfinal=a.ds, **a.args()), "extreme")


def test_values_that_are_not_numbers():
    """A NaN decay or key is in every later step of its head and in nothing before or beside it."""
    t = torch()
    announce("linattn NaN")
    for what in ("g", "k"):
        a = make((2, 140, 2, 2, 32, 32, "token", None, False), "f32", seed=15)
        clean = ssm.linattn(a.q, a.k, a.v, g=a.g)[0]
        bad = a.g.clone() if what == "g" else a.k.clone()
        bad[0, 70, 1] = float("nan")
        out = ssm.linattn(a.q, bad if what == "k" else a.k, a.v, g=bad if what == "g" else a.g)[0]
        assert out[0, 70:, 1].isnan().all()
        out[0, 70:, 1] = clean[0, 70:, 1]
        assert same(out, clean)


def test_empty():
    t = torch()
    announce("linattn empty")
    for b, L, h in ((0, 5, 2), (2, 0, 2), (2, 5, 0)):
        q, v = t.zeros(b, L, h, 8, device="cuda"), t.zeros(b, L, h, 4, device="cuda")
        s0 = t.randn(b, h, 4, 8, device="cuda")
        out, fin = ssm.linattn(q, q, v, initial_state=s0)
        assert out.shape == v.shape and same(fin, s0)
        g = t.zeros(h, device="cuda")
        d = ssm.linattn_backward(q, q, v, v, g, initial_state=s0, dfinal=s0)
        assert same(d["dinitial"], s0) and d["dg"].shape == (h,) and (d["dg"] == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_chained_calls(io):
    """A prompt in two calls, the state handed on, is one call; rows of no steps hand it on as it is."""
    announce(f"linattn chained {io}")
    a = make((2, 333, 1, 2, 64, 64, "token", None, True), io, seed=16)
    one = ssm.linattn(a.q, a.k, a.v, **a.args())
    first = ssm.linattn(a.q[:, :100], a.k[:, :100], a.v[:, :100], g=a.g[:, :100], initial_state=a.s0)
    second = ssm.linattn(a.q[:, 100:], a.k[:, 100:], a.v[:, 100:], g=a.g[:, 100:],
                         initial_state=first[1])
    check_forward(a, torch().cat((first[0], second[0]), 1), second[1], "chained")
    zero = torch().zeros(2, dtype=torch().int32, device="cuda")
    out, fin = ssm.linattn(a.q, a.k, a.v, g=a.g, initial_state=one[1], lengths=zero)
    assert same(fin, one[1]) and (out == 0).all()


def test_walked_states():
    """The backward's chunk states walked (past the caches) and joined (a few heads alone)."""
    t = torch()
    announce("linattn walked states")
    a = Attention(1, 2048, 16, 16, 128, 128, "bf16", "token", [1999], True, seed=17)
    assert ssm.ssm_linattn_bwd_workspace_bytes(1, 2048, 16, 128, 128, ssm.SSM_IO_BF16) > 64 << 20
    d = ssm.linattn_backward(a.q, a.k, a.v, a.dout, dfinal=a.ds, **a.args())
    h = slice(3, 5)
    e = ssm.linattn_backward(a.q[:, :, h], a.k[:, :, h], a.v[:, :, h], a.dout[:, :, h],
                             a.g[:, :, h].contiguous(), initial_state=a.s0[:, h].contiguous(),
                             lengths=a.n, dfinal=a.ds[:, h].contiguous())
    n = a.roundings * 2.0 ** -24
    for name in d:
        x, y = ((d[name][:, h], e[name]) if name == "dinitial" else (d[name][:, :, h], e[name]))
        x, y = x.double(), y.double()
        # each side is off by n roundings of terms whose 2-norm the result's stands for, and of bf16
        # results one more rounding each
        tol = 2 * n + (2 * 2.0 ** -8 if name in ("dq", "dk", "dv") else 0)
        assert (x - y).norm() <= tol * y.norm(), name


def test_long_segments():
    """Few heads over many chunks: segments side by side, against the same rows as a batch (whole)."""
    t = torch()
    announce("linattn segments")
    a = Attention(1, 9000, 1, 1, 64, 64, "f32", "token", None, True, seed=18)
    assert ssm.ssm_linattn_fwd_workspace_bytes(1, 9000, 1, 64, 64, ssm.SSM_IO_F32) > 0
    out, fin = ssm.linattn(a.q, a.k, a.v, **a.args())
    rows = lambda x: x.expand(400, *x.shape[1:])
    assert ssm.ssm_linattn_fwd_workspace_bytes(400, 9000, 1, 64, 64, ssm.SSM_IO_F32) == 0
    out2, fin2 = ssm.linattn(rows(a.q), rows(a.k), rows(a.v), g=rows(a.g),
                             initial_state=a.s0.expand(400, 1, 64, 64))
    n = 2 * a.roundings * 2.0 ** -24
    assert (out - out2[:1]).norm() <= n * out.norm() and (fin - fin2[399:]).norm() <= n * fin.norm()


def test_reproducible():
    announce("linattn reproducible")
    a = make((2, 300, 2, 8, 64, 64, "head", None, True), "bf16", seed=19)
    runs = [(*ssm.linattn(a.q, a.k, a.v, **a.args()),
             *ssm.linattn_backward(a.q, a.k, a.v, a.dout, dfinal=a.ds, **a.args()).values())
            for _ in range(3)]
    assert all(same(x, y) for r in runs[1:] for x, y in zip(r, runs[0]))


# ---------------------------------------------------------------- single tokens

def tokens(b, nslots, hk, h, dk, dv, io, decay, seed):
    r = Rand(seed)
    wide, wide64 = r((b, 2 * hk * dk + h * dv + 3), io)
    cut = lambda x, at, n, d: x[:, at:at + n * d].reshape(b, n, d)
    view = lambda x, at, n, d: x[:, at:at + n * d].unflatten(-1, (n, d))
    at = (1, 1 + hk * dk, 1 + 2 * hk * dk)
    sizes = ((hk, dk), (hk, dk), (h, dv))
    g, g64 = (None, None) if decay == "none" else r((h,) if decay == "head" else (b, h), "f32", 0.3)
    state, state64 = r((nslots, h, dv, dk))
    return ([view(wide, p, *s) for p, s in zip(at, sizes)],
            [cut(wide64, p, *s) for p, s in zip(at, sizes)], g, g64, state, state64)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(1, 1), (2, 3), (3, 16), (4, 64), (5, 7), (16, 33), (30, 20), (64, 64),
                                   (100, 50), (128, 128), (128, 64), (255, 9), (256, 256)])
def test_step(dk, dv, io):
    t = torch()
    for b, hk, h, decay, slots in ((1, 1, 1, "none", None), (3, 2, 4, "token", [4, 0, 2]),
                                   (5, 1, 3, "head", [1, -1, 1, 6, 1])):
        announce(f"linattn_step b{b} h{h} {dk}x{dv} {io} {slots}")
        (q, k, v), (q64, k64, v64), g, g64, state, state64 = tokens(b, 6, hk, h, dk, dv, io, decay, 30 + dk)
        s = None if slots is None else t.tensor(slots, dtype=t.int32, device="cuda")
        out = ssm.linattn_step(q, k, v, state, g, slots=s)
        ref, after = ol.linattn_step_ref(q64, k64, v64, state64, g64, slots=slots)
        ab, aafter = ol.linattn_step_ref(*map(np.abs, (q64, k64, v64, state64)), g64, slots=slots)
        n = roundings(dk, dv, 1)
        within(out, ref, ab, io, n, "step out", pairs=False)
        within(state, after, aafter, "f32", n, "step state")


def test_step_many():
    """Enough rows for many states a lane, through and past the caches."""
    t = torch()
    for b, h, dk, dv in ((600, 16, 128, 64), (64, 33, 64, 100)):
        announce(f"linattn_step many b{b} h{h} {dk}x{dv}")
        (q, k, v), _, g, _, state, _ = tokens(b, 2, 1, h, dk, dv, "bf16", "token", 40)
        state = t.randn(b + 5, h, dv, dk, device="cuda")
        before, slots = state.double(), t.randperm(b + 5, device="cuda")[:b].to(t.int32)
        out = ssm.linattn_step(q, k, v, state, g, slots=slots)
        at = slots.long()
        want = before.clone()
        want[at] = want[at] * g.double().exp()[:, :, None, None] + v.double()[..., None] * k.double()[:, :, None]
        assert (state.double() - want).norm() <= 8 * 2.0 ** -24 * want.norm()
        o = (want[at] * q.double()[:, :, None]).sum(3) * dk ** -0.5
        assert (out.double() - o).norm() <= (2.0 ** -8 + dk * 2.0 ** -24) * o.norm()
        rest = t.ones(b + 5, dtype=t.bool, device="cuda")
        rest[at] = False
        assert t.equal(state[rest].double(), before[rest])


def test_step_large_cache():
    t = torch()
    nslots = 70000  # of 32768 states: 2.3e9 floats
    announce("linattn_step large cache")
    state = t.empty(nslots, 1, 256, 128, device="cuda")
    slots = [nslots - 1, 0, 65536]
    state[slots] = t.randn(3, 1, 256, 128, device="cuda")
    (q, k, v), (q64, k64, v64), g, g64, _, _ = tokens(3, 1, 1, 1, 128, 256, "f32", "token", 41)
    small = state[slots].clone()
    ref, after = ol.linattn_step_ref(q64, k64, v64, host(small), g64)
    out = ssm.linattn_step(q, k, v, state, g, slots=t.tensor(slots, dtype=t.int32, device="cuda"))
    ab, aafter = ol.linattn_step_ref(*map(np.abs, (q64, k64, v64, host(small))), g64)
    within(out, ref, ab, "f32", roundings(128, 256, 1), "large out")
    within(state[slots], after, aafter, "f32", roundings(128, 256, 1), "large state")


def test_steps_are_the_prompt():
    t = torch()
    announce("linattn steps are the prompt")
    a = make((3, 70, 2, 4, 48, 40, "token", None, True), "f32", seed=42)
    cache, slots = t.zeros(5, 4, 40, 48, device="cuda"), t.tensor([3, 0, 4], dtype=t.int32, device="cuda")
    cache[slots.long()] = a.s0
    out = t.stack([ssm.linattn_step(a.q[:, i], a.k[:, i], a.v[:, i], cache, a.g[:, i], slots=slots)
                   for i in range(70)], 1)
    check_forward(a, out, cache[slots.long()], "steps")
