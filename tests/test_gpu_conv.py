"""GPU parity of the short causal convolution (conv, conv_backward, causal_conv, conv_step)
against the float64 oracle (oracle/block.py, pinned in test_oracle_block_pins.py).

Shapes cover: one step, sequences shorter than the window, of one lane's 8 steps, of a wave's
64 x 8 steps and either side of both, ragged tails, channel counts that are no multiple of a
16-byte word or of a wave's 64 channels; x with steps or with channels contiguous, aligned
and at odd addresses; every optional input; rows that end early, at once, and past the end.
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import TOL, Rand, check, dtype, ordered, same, sum_tol
from gpu_util import announce, host, torch
from oracle import block as ob

pytestmark = pytest.mark.gpu

SHAPES = [
    # (batch, dim, seqlen, width)
    (1, 1, 1, 4), (2, 3, 2, 4), (3, 5, 3, 2), (2, 64, 7, 3), (2, 72, 8, 4), (1, 130, 9, 4),
    (2, 33, 63, 4), (2, 64, 64, 4), (1, 65, 65, 2), (2, 40, 255, 3), (1, 24, 513, 4),
    (3, 67, 777, 4), (1, 16, 2053, 4), (1, 7, 4500, 3),
]
ids = lambda s: "b{}d{}L{}W{}".format(*s)


def make(shape, io, seed, state=True):
    b, d, L, w = shape
    r = Rand(seed)
    return {"x": r((b, d, L), io), "weight": r((d, w), scale=0.5), "bias": r((d,), scale=0.5),
            "init": r((b, d, w - 1), io), "dout": r((b, d, L), io), "dfinal": r((b, d, w - 1), io)}


def lengths_of(b, L, seed):
    """Some row of every kind: whole, empty, shorter than the window, past the end, negative."""
    kinds = [L, 0, min(1, L), L + 7, -3, L // 2, max(L - 1, 0)]
    n = [kinds[(seed + i) % len(kinds)] for i in range(b)]
    return n, torch().tensor(n, dtype=torch().int32, device="cuda")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["time", "channel", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_conv_forward(shape, order, io):
    b, d, L, w = shape
    for k, (silu, bias, init, lens) in enumerate([(True, True, True, True),
                                                  (False, False, False, False)]):
        announce(f"conv forward {ids(shape)} {order} {io} variant {k}")
        v = make(shape, io, 100 + L + w)
        n, lengths = lengths_of(b, L, k + L) if lens else (None, None)
        pick = lambda name, on: v[name] if on else (None, None)
        out, fin = ssm.conv(ordered(v["x"][0], order), v["weight"][0], bias=pick("bias", bias)[0],
                            silu=silu, initial_state=pick("init", init)[0], lengths=lengths)
        ref, rfin = ob.conv_ref(v["x"][1], v["weight"][1], pick("bias", bias)[1], silu,
                                pick("init", init)[1], n)
        check(out, ref, TOL[io], "out")
        assert out.is_contiguous() and np.array_equal(host(fin), rfin)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["time", "channel", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_conv_backward(shape, order, io):
    b, d, L, w = shape
    for k, (silu, full) in enumerate([(True, True), (False, False)]):
        announce(f"conv backward {ids(shape)} {order} {io} variant {k}")
        v = make(shape, io, 200 + L + w)
        n, lengths = lengths_of(b, L, k + L) if full else (None, None)
        pick = lambda name: v[name] if full else (None, None)
        x = ordered(v["x"][0], order)
        g = ssm.conv_backward(x, v["weight"][0], v["dout"][0], bias=pick("bias")[0], silu=silu,
                              initial_state=pick("init")[0], lengths=lengths,
                              dfinal=pick("dfinal")[0])
        ref = ob.conv_bwd_ref(v["x"][1], v["weight"][1], v["dout"][1], pick("bias")[1], silu,
                              pick("init")[1], n, pick("dfinal")[1])
        check(g["dx"], ref["dx"], TOL[io], "dx")
        check(g["dweight"], ref["dweight"], sum_tol(b * L), "dweight")
        if full:
            check(g["dbias"], ref["dbias"], sum_tol(b * L), "dbias")
            check(g["dinitial"], ref["dinitial"], TOL[io], "dinitial")
        else:
            assert g["dbias"] is None and g["dinitial"] is None
        if L > 1 and d > 1:
            assert g["dx"].stride(2 if order == "time" else 1) == 1


@pytest.mark.parametrize("order", ["time", "channel"])
def test_conv_reads_nothing_behind_a_row(order):
    """NaN and infinities at and behind each row's end, in x and in dout, change nothing."""
    announce(f"conv poisoned tails {order}")
    shape = (4, 70, 100, 4)
    v = make(shape, "bf16", 300)
    n = [100, 37, 2, 0]
    lengths = torch().tensor(n, dtype=torch().int32, device="cuda")
    x, dout = v["x"][0].clone(), v["dout"][0].clone()
    for i, e in enumerate(n):
        x[i, :, e:] = float("nan")
        x[i, ::2, e:] = float("inf")
        dout[i, :, e:] = float("nan")
    args = dict(bias=v["bias"][0], silu=True, initial_state=v["init"][0], lengths=lengths)
    a, fa = ssm.conv(ordered(x, order), v["weight"][0], **args)
    b, fb = ssm.conv(ordered(v["x"][0], order), v["weight"][0], **args)
    assert same(a, b) and same(fa, fb)
    ga = ssm.conv_backward(ordered(x, order), v["weight"][0], dout, dfinal=v["dfinal"][0], **args)
    gb = ssm.conv_backward(ordered(v["x"][0], order), v["weight"][0], v["dout"][0],
                           dfinal=v["dfinal"][0], **args)
    for k in ga:
        assert same(ga[k].contiguous(), gb[k].contiguous()), k
    assert not host(a)[3].any() and not host(ga["dx"])[3].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_nonfinite_inputs_stay_in_their_window(io):
    announce(f"conv NaN window {io}")
    t = torch()
    v = make((1, 66, 300, 4), io, 310)
    x = v["x"][0].clone()
    x[0, 65, 150] = float("nan")
    x[0, 3, 20] = float("inf")
    for order in ("time", "channel"):
        out, _ = ssm.conv(ordered(x, order), v["weight"][0])
        bad = ~t.isfinite(out)
        want = t.zeros_like(bad)
        want[0, 65, 150:154] = True
        want[0, 3, 20:24] = True
        assert t.equal(bad, want), order


def test_conv_empty():
    announce("conv empty")
    t = torch()
    w = t.randn(5, 4, device="cuda")
    init = t.randn(2, 5, 3, device="cuda")
    x = t.empty(2, 5, 0, device="cuda")
    out, fin = ssm.conv(x, w, initial_state=init)
    assert out.shape == (2, 5, 0) and same(fin, init)
    _, fin = ssm.conv(x, w)
    assert not fin.any()
    df = t.randn(2, 5, 3, device="cuda")
    g = ssm.conv_backward(x, w, x, bias=w[:, 0].contiguous(), initial_state=init, dfinal=df)
    assert same(g["dinitial"], df) and not g["dweight"].any() and not g["dbias"].any()
    g = ssm.conv_backward(t.empty(0, 5, 8, device="cuda"), w, t.empty(0, 5, 8, device="cuda"))
    assert not g["dweight"].any()
    out, fin = ssm.conv(t.empty(0, 5, 8, device="cuda"), w)
    assert out.shape == (0, 5, 8) and fin.shape == (0, 5, 3)


def test_conv_batch_inside_time_and_broadcast_rows():
    """Orders beside the usual two: a [seqlen, batch, dim] buffer, one row for all of a batch."""
    announce("conv other strides")
    t = torch()
    r = Rand(320)
    w, w64 = r((24, 4))
    x, x64 = r((50, 3, 24), "bf16")
    out, _ = ssm.conv(x.permute(1, 2, 0), w)
    check(out, ob.conv_ref(x64.transpose(1, 2, 0), w64)[0], TOL["bf16"], "[L, B, D]")
    row, row64 = r((1, 24, 90), "bf16")
    out, _ = ssm.conv(row.expand(3, 24, 90), w)
    ref = np.repeat(ob.conv_ref(row64, w64)[0], 3, axis=0)
    check(out, ref, TOL["bf16"], "expanded")
    g = ssm.conv_backward(row.expand(3, 24, 90), w, out)
    gref = ob.conv_bwd_ref(np.repeat(row64, 3, axis=0), w64, host(out))
    check(g["dx"], gref["dx"], TOL["bf16"], "expanded dx")
    every_second = t.randn(2, 24, 120, device="cuda")[:, :, ::2]  # copied: neither contiguous
    out, _ = ssm.conv(every_second, w)
    check(out, ob.conv_ref(host(every_second), w64)[0], TOL["f32"], "every second step")


@pytest.mark.parametrize("order", ["time", "channel"])
def test_conv_layer_size(order):
    """The convolution ahead of the Mamba-2 layer (b4, 2048 + 2 x 128 channels, 2048 steps):
    both directions on sampled channels against the oracle, and bitwise reproducible."""
    announce(f"conv layer {order}")
    t = torch()
    shape = (4, 2304, 2048, 4)
    g = t.Generator(device="cuda").manual_seed(5)
    x = ordered(t.randn(shape[:3], device="cuda", generator=g).bfloat16(), order)
    dout = t.randn(shape[:3], device="cuda", generator=g).bfloat16()
    w, bias = t.randn(2304, 4, device="cuda", generator=g), t.randn(2304, device="cuda", generator=g)
    out, fin = ssm.conv(x, w, bias=bias, silu=True)
    grads = ssm.conv_backward(x, w, dout, bias=bias, silu=True)
    at = [0, 7, 8, 63, 64, 1000, 2047, 2048, 2303]
    pick = lambda v: host(v[:, at].contiguous())
    rout, rfin = ob.conv_ref(pick(x), host(w[at]), host(bias[at]), True)
    check(pick(out), rout, TOL["bf16"], "out")
    assert np.array_equal(pick(fin), rfin)
    ref = ob.conv_bwd_ref(pick(x), host(w[at]), pick(dout), host(bias[at]), True)
    check(pick(grads["dx"]), ref["dx"], TOL["bf16"], "dx")
    check(grads["dweight"][at], ref["dweight"], sum_tol(4 * 2048), "dweight")
    check(grads["dbias"][at], ref["dbias"], sum_tol(4 * 2048), "dbias")
    again = ssm.conv_backward(x, w, dout, bias=bias, silu=True)
    assert all(same(grads[k].contiguous(), again[k].contiguous()) for k in ("dx", "dweight", "dbias"))


def test_causal_conv_autograd():
    announce("causal_conv autograd")
    t = torch()
    v = make((2, 20, 90, 4), "f32", 330)
    leaf = {k: v[k][0].clone().requires_grad_() for k in ("x", "weight", "bias", "init")}
    lengths = t.tensor([90, 31], dtype=t.int32, device="cuda")
    out, fin = ssm.causal_conv(leaf["x"], leaf["weight"], leaf["bias"], True, leaf["init"], lengths)
    ((out * v["dout"][0]).sum() + (fin * v["dfinal"][0]).sum()).backward()
    ref = ob.conv_bwd_ref(v["x"][1], v["weight"][1], v["dout"][1], v["bias"][1], True, v["init"][1],
                          [90, 31], v["dfinal"][1])
    for name, key in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("init", "dinitial")):
        check(leaf[name].grad, ref[key], sum_tol(180), key)
    # only the final state used, and no initial state or bias
    x, w = v["x"][0].clone().requires_grad_(), v["weight"][0].clone().requires_grad_()
    ssm.causal_conv(x, w)[1].sum().backward()
    assert float(x.grad[:, :, -3:].sum()) == 2 * 20 * 3 and not x.grad[:, :, :-3].any()
    assert not w.grad.any()


# ---------------------------------------------------------------- single tokens

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("bd", [(1, 1), (3, 7), (8, 64), (5, 515), (70, 2304), (2, 6000)],
                         ids=lambda s: "b{}d{}".format(*s))
def test_conv_step(bd, width, io):
    b, d = bd
    announce(f"conv_step b{b} d{d} W{width} {io}")
    t = torch()
    r = Rand(400 + b + d + width)
    wide, wide64 = r((b, d + 9), io)
    x, x64 = wide[:, 3:3 + d], wide64[:, 3:3 + d]
    w, w64 = r((d, width))
    bias, bias64 = r((d,))
    for slots in (None, list(range(b))[::-1], [(7 * i) % (b + 5) - 2 for i in range(b)]):
        n = b if slots is None else b + 3
        state, s64 = r((n, d, width - 1), io)
        s = None if slots is None else t.tensor(slots, dtype=t.int32, device="cuda")
        out = ssm.conv_step(x, state, w, bias=bias, silu=True, slots=s)
        ref, after = ob.conv_step_ref(x64, s64, w64, bias64, True, slots)
        check(out, ref, TOL[io], f"out {slots is None}")
        assert np.array_equal(host(state), after)


def test_conv_step_rows_of_one_slot():
    """Every row names the same slot: successive tokens; and a mixture with rows of no slot."""
    announce("conv_step repeated slots")
    t = torch()
    r = Rand(410)
    for slots in ([2] * 9, [0, 2, 0, -1, 2, 2, 99, 0, 1], [1] * 200 + [3] + [1] * 3):
        x, x64 = r((len(slots), 40), "bf16")
        state, s64 = r((4, 40, 3), "bf16")
        w, w64 = r((40, 4))
        out = ssm.conv_step(x, state, w, slots=t.tensor(slots, dtype=t.int32, device="cuda"))
        ref, after = ob.conv_step_ref(x64, s64, w64, slots=slots)
        check(out, ref, TOL["bf16"], f"{len(slots)} rows")
        assert np.array_equal(host(state), after)


def test_conv_step_empty():
    announce("conv_step empty")
    t = torch()
    out = ssm.conv_step(t.empty(0, 8, device="cuda"), t.zeros(2, 8, 3, device="cuda"),
                        t.zeros(8, 4, device="cuda"))
    assert out.shape == (0, 8)
    out = ssm.conv_step(t.ones(2, 8, device="cuda"), t.zeros(0, 8, 3, device="cuda"),
                        t.zeros(8, 4, device="cuda"),
                        slots=t.zeros(2, dtype=t.int32, device="cuda"))
    assert not out.any()
