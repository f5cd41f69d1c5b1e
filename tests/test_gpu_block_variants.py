"""The launch forms that the operators around the scan take only past a size: two rows a lane of the
convolution step, two tiles a wave of the convolution in time order, the state step's forms by
channels a lane and past the caches, the norm's sixteen waves and its two launches with a result
in time order. Each against the float64 oracle, on sampled channels, rows or tokens (channels of
the convolution and the state step, and tokens of the norm, do not meet). That the sizes here take
those forms is checked on the CPU (test_block_launch_rules.py).
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import TOL, check, dtype, ordered
from gpu_util import announce, host, torch
from oracle import block as ob
from ssm_workloads import WATCH

pytestmark = pytest.mark.gpu

# One product, one sum and a decay whose exponent's rounding is |dt A log2 e| 2^-24 of a factor
# of at most one, per step of a slot; a slot here takes at most four steps: under 4 * 40 * 2^-24
# of the metric's |r| + rms.
STATE_TOL = 1e-5


def chain_tol(chain, n):
    """A float32 sum of n random terms with at most `chain` roundings on a term's way, each 2^-24
    of an absolute sum about sqrt(n) times the rms of the signed one; and the terms' own error."""
    return chain * 2.0 ** -24 * max(n, 1) ** 0.5 + TOL["f32"]


def draws(seed):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return lambda *s, io="f32": t.randn(s, device="cuda", generator=g).to(dtype(io))


def slots_of(b, nslots, shift):
    """Most rows a slot of their own; neighbours and far rows that share one, four rows of one,
    rows of none, out of range."""
    s = [(i * 7 + shift) % nslots for i in range(b)]  # (7 and nslots share no factor)
    s[1] = s[0]
    s[6], s[7], s[b - 1] = s[5], s[5], s[5]
    s[b // 2] = s[3]
    s[10], s[11], s[b - 4] = -1, nslots, -5
    return s


# ---------------------------------------------------------------- convolution step

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("d", [6000, 6001])
def test_conv_step_two_rows(d, width, io):
    b, nslots = 385, 401
    announce(f"conv_step b{b} d{d} W{width} {io}")
    t, mk = torch(), draws(800 + d + width)
    x, w, bias = mk(b, d + 9, io=io)[:, 3:3 + d], mk(d, width), mk(d)
    at = [0, 1, 2, 3, 511, 512, 1023, 1024, 3001, d - 2, d - 1]
    pick = lambda v: host(v[:, at].contiguous())
    for slots in (None, slots_of(b, nslots, width)):
        state = mk(nslots, d, width - 1, io=io)
        before = pick(state)
        s = None if slots is None else t.tensor(slots, dtype=t.int32, device="cuda")
        out = ssm.conv_step(x, state, w, bias=bias, silu=True, slots=s)
        ref, after = ob.conv_step_ref(pick(x), before, host(w[at]), host(bias[at]), True, slots)
        check(pick(out), ref, TOL[io], f"out {slots is None}")
        assert np.array_equal(pick(state), after)


# ---------------------------------------------------------------- convolution, time order

@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("shape", [(3, 2731, 777), (2, 8200, 500), (16, 6000, 100), (2, 2741, 1531),
                                   (1, 4099, 2048)],
                         ids=lambda s: "b{}d{}L{}".format(*s))
def test_conv_tiles(shape, width):
    """Rows of one, two, three and four tiles where the waves fill the device, with lengths that end
    in each tile and an initial state."""
    b, d, L = shape
    announce(f"conv tiles b{b} d{d} L{L} W{width}")
    t, mk = torch(), draws(820 + L + width)
    x, w, bias = mk(b, d, L, io="bf16"), mk(d, width), mk(d)
    init = mk(b, d, width - 1, io="bf16")
    n = [[L, L // 3, 0, 1, L + 3, max(L - 515, 0), L - 1][(i + width) % 7] for i in range(b)]
    lengths = t.tensor(n, dtype=t.int32, device="cuda")
    at = [0, 1, 63, 64, 777, d - 2, d - 1]
    pick = lambda v: host(v[:, at].contiguous())
    for full in (True, False):
        opt = dict(initial_state=init, lengths=lengths) if full else {}
        out, fin = ssm.conv(x, w, bias=bias, silu=True, **opt)
        ref, rfin = ob.conv_ref(pick(x), host(w[at]), host(bias[at]), True,
                                pick(init) if full else None, n if full else None)
        check(pick(out), ref, TOL["bf16"], f"out {full}")
        assert np.array_equal(pick(fin), rfin)


# ---------------------------------------------------------------- state step

# (rows, channels, states, heads): Mamba-1 through the caches, its states no whole words, past the
# caches; Mamba-2 likewise.
STEPS = [(256, 2560, 16, None), (250, 5000, 5, None), (250, 4099, 7, None), (256, 4100, 33, None),
         (40, 4096, 128, 32), (128, 4096, 64, 64), (100, 4096, 100, 64), (200, 6144, 128, 48)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", STEPS, ids=lambda s: "b{}d{}N{}h{}".format(*s))
def test_state_step_forms(case, io):
    b, d, n, heads = case
    announce(f"state step b{b} d{d} N{n} heads {heads} {io}")
    t, mk = torch(), draws(840 + b + d + n)
    nslots = b + 1 if (b + 1) % 7 else b + 2
    row = mk(b, d + 2 * n + 1, io=io)
    x, B, C = row[:, 1:1 + d], row[:, 1 + d:1 + d + n], row[:, 1 + d + n:]
    z, D, steps = mk(b, d, io=io), mk(d), d if heads is None else heads
    dt, bias = 0.5 * mk(b, steps, io=io), mk(steps)
    A = -mk(d, n).abs() - 0.1 if heads is None else -mk(heads).abs() - 0.1
    state = mk(nslots, d, n)
    slots = slots_of(b, nslots, n)
    s = t.tensor(slots, dtype=t.int32, device="cuda")
    if heads is None:  # sampled channels, or all channels of sampled heads
        pick_steps = at = [0, 1, 15, 16, 63, 64, 1000, d - 2, d - 1]
    else:
        pick_steps = [0, 1, heads - 1]
        at = [h * (d // heads) + i for h in pick_steps for i in range(d // heads)]
    before = host(state[:, at])
    opt = dict(D=D, z=z, slots=s)
    if heads is None:
        out = ssm.scan_step(x, dt, A, B, C, state, delta_bias=bias, delta_softplus=True, **opt)
    else:
        out = ssm.ssd_step(x, dt, A, B, C, state, dt_bias=bias, dt_softplus=True, **opt)
    ref, after = ob.step_ref(host(x[:, at].contiguous()), host(dt[:, pick_steps].contiguous()), host(A[pick_steps]),
                             host(B.contiguous()), host(C.contiguous()), before, host(D[at]),
                             host(z[:, at].contiguous()), host(bias[pick_steps]), True, slots)
    check(out[:, at].contiguous(), ref, max(1e-4, WATCH[io] if io == "bf16" else 0), "out")
    check(state[:, at], after, STATE_TOL, "state")


# ---------------------------------------------------------------- norm

# (io, batch, channels, steps): sixteen waves; two launches for odd rows; for a group that does
# not fit.
NORMS = [("f32", 4, 2048, 2047), ("f32", 4, 2048, 2048), ("bf16", 4, 4096, 1021), ("bf16", 1, 4096, 1023),
         ("bf16", 1, 8200, 9), ("f32", 1, 5001, 77)]


@pytest.mark.parametrize("mode", ["none", "gate_first", "norm_first"])
@pytest.mark.parametrize("case", NORMS, ids=lambda s: "{}-b{}d{}L{}".format(*s))
def test_norm_forms(case, mode):
    io, b, d, L = case
    announce(f"norm forms {case} {mode}")
    mk = draws(860 + d + L)
    y, w = mk(b, d, L, io=io), mk(d)
    z = None if mode == "none" else ordered(mk(b, d, L, io=io), "channel")
    first = mode == "norm_first"
    at = sorted({0, 1, 7, 8 % L, L // 2, L - 9 if L > 9 else 0, L - 2, L - 1})
    pick = lambda v: None if v is None else host(v[:, :, at].contiguous())
    out, rstd = ssm.norm_train(y, w, z=z, norm_before_gate=first)
    ref, rref = ob.norm_ref(pick(y), host(w), pick(z), 1e-5, 1, first)
    check(pick(out), ref, TOL[io], "out")
    assert np.abs(pick(rstd) / rref - 1).max() <= 64 * 2.0 ** -24
    dout = mk(b, d, L, io=io)
    g = ssm.norm_backward(y, w, rstd, dout, z=z, norm_before_gate=first)
    gref = ob.norm_bwd_ref(pick(y), host(w), pick(dout), pick(z), 1e-5, 1, first)
    check(pick(g["dy"]), gref["dy"], TOL[io], "dy")
    if z is not None:
        check(pick(g["dz"]), gref["dz"], TOL[io], "dz")
    # dweight needs every token: in float64 on the device
    yd, gd = y.double(), dout.double()
    gate = 1.0 if z is None else z.double() * z.double().sigmoid()
    v = yd if first else yd * gate
    n = v * ((v * v).mean(1, keepdim=True) + 1e-5).rsqrt()
    dw = ((gd * gate if first else gd) * n).sum((0, 2))
    # a lane's 4 steps, 6 adds across lanes, partial rows (of 8 steps at least) in 32 slices
    chain = 4 + 6 + b * L // 8 // 32 + 1 + 32
    check(g["dweight"], dw.cpu().numpy(), chain_tol(chain, b * L), "dweight")
