"""GPU parity of the single-token state steps (scan_step, ssd_step) against the float64 oracle
(oracle/block.py, pinned in test_oracle_block_pins.py).

Cover: states from 1 to 256 with and without whole 16-byte words; channel counts that leave a
wave partly idle; rows of larger tensors; slots in any order, missing, out of range, repeated;
a cache of more than 2^31 states; non-finite values in one row.
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import Rand, check, same
from gpu_util import announce, host, torch
from oracle import block as ob
from ssm_workloads import RTOL, WATCH

pytestmark = pytest.mark.gpu

# The state: one product and one sum in float32, and exp2's argument rounded, |dt A log2 e|
# 2^-24 of a factor that is at most one: under 1e-5 of the metric's |r| + rms.
STATE_TOL = 1e-5


def make(b, dim, n, heads, io, nslots, seed):
    """Rows cut out of one wider row, as a convolution's output is cut."""
    r = Rand(seed)
    wide, wide64 = r((b, dim + 2 * n + 3), io)
    cut = lambda lo, k: (wide[:, lo:lo + k], wide64[:, lo:lo + k])
    steps = dim if heads is None else heads
    A, A64 = r((dim, n) if heads is None else (heads,))
    return {"x": cut(1, dim), "B": cut(1 + dim, n), "C": cut(1 + dim + n, n),
            "dt": r((b, steps), io, 0.5), "A": (-A.abs() - 0.1, -np.abs(A64) - 0.1),
            "D": r((dim,)), "z": r((b, dim), io), "bias": r((steps,)), "state": r((nslots, dim, n))}


def run(v, heads, slots=None, full=True, softplus=True):
    t = torch()
    s = None if slots is None else t.tensor(slots, dtype=t.int32, device="cuda")
    opt = lambda k: v[k][0] if full else None
    opt64 = lambda k: v[k][1] if full else None
    a = [v[k][0] for k in ("x", "dt", "A", "B", "C", "state")]
    # the float32 value of A on both sides: -|a| - 0.1 is rounded on the device
    A64 = host(v["A"][0])
    if heads is None:
        out = ssm.scan_step(*a, D=opt("D"), z=opt("z"), delta_bias=opt("bias"),
                            delta_softplus=softplus, slots=s)
    else:
        out = ssm.ssd_step(*a, D=opt("D"), z=opt("z"), dt_bias=opt("bias"), dt_softplus=softplus,
                           slots=s)
    ref, after = ob.step_ref(v["x"][1], v["dt"][1], A64, v["B"][1], v["C"][1], v["state"][1],
                             opt64("D"), opt64("z"), opt64("bias"), softplus, slots)
    return out, ref, after


def compare(io, v, out, ref, after, label):
    check(out, ref, max(RTOL["f32"], WATCH[io] if io == "bf16" else 0), label + " out")
    check(v["state"][0], after, STATE_TOL, label + " state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 16, 30, 64, 100, 128, 255, 256])
def test_scan_step(n, io):
    for b, dim in ((1, 1), (3, 70), (5, 515)):
        announce(f"scan_step b{b} d{dim} N{n} {io}")
        v = make(b, dim, n, None, io, b + 2, 500 + n + dim)
        out, ref, after = run(v, None, [(i * 2 + 1) % (b + 2) for i in range(b)], full=dim != 70)
        compare(io, v, out, ref, after, f"N{n} d{dim}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64), (2, 3, 16, 128), (4, 5, 48, 100), (8, 32, 64, 128),
                                   (3, 2, 7, 256), (2, 4, 128, 16)],
                         ids=lambda s: "b{}h{}x{}N{}".format(*s))
def test_ssd_step(shape, io):
    b, heads, p, n = shape
    announce(f"ssd_step {shape} {io}")
    for full, softplus in ((True, True), (False, False)):
        v = make(b, heads * p, n, heads, io, b, 520 + n + p)
        if not softplus:  # positive step sizes
            v["dt"] = (v["dt"][0].abs(), np.abs(v["dt"][1]))
        out, ref, after = run(v, heads, None, full, softplus)
        compare(io, v, out, ref, after, f"{shape} {full}")


@pytest.mark.parametrize("heads", [None, 4])
def test_step_slots(heads):
    """Rows of no slot are zero and change nothing; rows of one slot are successive tokens."""
    for slots in ([3, -1, 0, 7, 2], [1, 1, 1, 1], [0, 2, 0, -5, 2, 2, 4, 0], [1] * 70 + [0, 1]):
        announce(f"step slots {slots[:8]} of {len(slots)} heads {heads}")
        v = make(len(slots), 80, 16, heads, "bf16", 5, 540 + len(slots))
        out, ref, after = run(v, heads, slots)
        compare("bf16", v, out, ref, after, "slots")
        untouched = [s for s in range(5) if s not in slots]
        assert np.array_equal(host(v["state"][0])[untouched], v["state"][1][untouched])
        for i, s in enumerate(slots):
            if not 0 <= s < 5:
                assert not out[i].any()


def test_step_matches_the_scan_of_one_step():
    """scan_step against scan with seqlen 1 and the state handed in (the short kernel)."""
    announce("scan_step against scan")
    v = make(4, 200, 16, None, "bf16", 4, 560)
    g = {k: v[k][0].contiguous() for k in v}
    one = lambda t: t.unsqueeze(2)
    want, fin = ssm.scan(one(g["x"]), one(g["dt"]), g["A"], one(g["B"]), one(g["C"]), D=g["D"],
                         z=one(g["z"]), delta_bias=g["bias"], delta_softplus=True,
                         h0=v["state"][0])
    out, ref, after = run(v, None)
    check(fin, after, STATE_TOL, "scan state")
    check(v["state"][0], after, STATE_TOL, "step state")
    check(out, host(want)[:, :, 0], WATCH["bf16"] * 2, "out of both")


def test_step_cache_past_32_bits():
    """Slots whose offsets pass 2^31 states (2^33 bytes)."""
    announce("step large cache")
    t = torch()
    dim, n = 4096, 128
    nslots = (1 << 31) // (dim * n) + 3
    state = t.empty((nslots, dim, n), device="cuda")
    slots = [nslots - 1, 1, nslots - 2]
    v = make(3, dim, n, 64, "bf16", 3, 570)
    for i, s in enumerate(slots):
        state[s] = v["state"][0][i]
    guard = state[nslots - 3].fill_(7.0).clone()
    small = v["state"]
    out_small, ref, after = run(v, 64)
    v["state"] = (state, None)
    s = t.tensor(slots, dtype=t.int32, device="cuda")
    out = ssm.ssd_step(*(v[k][0] for k in ("x", "dt", "A", "B", "C", "state")), D=v["D"][0],
                       z=v["z"][0], dt_bias=v["bias"][0], dt_softplus=True, slots=s)
    assert same(out, out_small)
    for i, k in enumerate(slots):
        assert same(state[k], small[0][i])
    assert same(state[nslots - 3], guard)
    check(out, ref, WATCH["bf16"], "out")


@pytest.mark.parametrize("heads,dim,n,b", [(None, 5617, 100, 70), (64, 4288, 30, 290)])
def test_step_states_past_the_caches(heads, dim, n, b):
    """More states than the caches hold (128 MiB and more): every row as in calls of a few
    rows, which take another variant, bit for bit, repeated and missing slots among them; and
    two of them against the oracle."""
    announce(f"step of {b * dim * n * 4 >> 20} MiB of states, heads {heads}")
    t = torch()
    v = make(b, dim, n, heads, "bf16", 3, 575)
    state = v["state"][0].repeat((b + 2) // 3 + 2, 1, 1)
    nslots = state.shape[0]
    slots = [(i * 7 + 3) % nslots for i in range(b)]
    slots[5], slots[b - 1], slots[9] = slots[2], slots[2], -1
    entry = ssm.scan_step if heads is None else ssm.ssd_step
    names = ("delta_bias", "delta_softplus") if heads is None else ("dt_bias", "dt_softplus")

    def call(lo, hi, st):
        r = {k: v[k][0][lo:hi] for k in ("x", "dt", "B", "C", "z")}
        return entry(r["x"], r["dt"], v["A"][0], r["B"], r["C"], st, D=v["D"][0], z=r["z"],
                     slots=t.tensor(slots[lo:hi], dtype=t.int32, device="cuda"),
                     **dict(zip(names, (v["bias"][0], True))))
    few = state.clone()
    parts = t.cat([call(lo, min(lo + 10, b), few) for lo in range(0, b, 10)])
    out = call(0, b, state)
    assert same(out, parts) and same(state, few)
    rows = [1, b - 2]
    assert slots.count(slots[1]) == slots.count(slots[b - 2]) == 1
    before = v["state"][1][[slots[i] % 3 for i in rows]]
    ref, after = ob.step_ref(*(v[k][1][rows] for k in ("x", "dt")), host(v["A"][0]),
                             v["B"][1][rows], v["C"][1][rows], before, v["D"][1],
                             v["z"][1][rows], v["bias"][1], True, None)
    check(out[rows], ref, WATCH["bf16"], "out")
    check(state[[slots[i] for i in rows]], after, STATE_TOL, "state")


def test_step_nonfinite_rows_stay_apart():
    announce("step non-finite")
    t = torch()
    v = make(4, 130, 20, None, "f32", 4, 580)
    x = v["x"][0].clone()
    x[2, 5] = float("inf")
    a = [v[k][0] for k in ("dt", "A", "B", "C")]
    clean_state = v["state"][0].clone()
    clean = ssm.scan_step(v["x"][0], *a, clean_state, delta_softplus=True)
    state = v["state"][0].clone()
    out = ssm.scan_step(x, *a, state, delta_softplus=True)
    bad = ~t.isfinite(out)
    assert bad[2, 5] and int(bad.sum()) == 1
    keep = t.ones_like(bad)
    keep[2, 5] = False
    assert same(out[keep], clean[keep]) and same(state[keep], clean_state[keep])
    assert bool((~t.isfinite(state[2, 5])).all())


def test_step_empty():
    announce("step empty")
    t = torch()
    z = lambda *s: t.zeros(*s, device="cuda")
    assert ssm.scan_step(z(0, 8), z(0, 8), z(8, 4), z(0, 4), z(0, 4), z(2, 8, 4)).shape == (0, 8)
    out = ssm.ssd_step(z(2, 8) + 1, z(2, 2), z(2), z(2, 4), z(2, 4), z(0, 8, 4),
                       slots=t.zeros(2, dtype=t.int32, device="cuda"))
    assert not out.any()
