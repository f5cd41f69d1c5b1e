"""GPU parity of the gated RMS norm (norm, norm_train, norm_backward, gated_norm) against the
float64 oracle (oracle/block.py, pinned in test_oracle_block_pins.py).

Cover: every memory order of y, z and out; groups from a few channels to more than a
workgroup holds at once; channel and step counts that are no multiple of a lane's square;
single tokens; rows of zeros; large and small magnitudes.
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import TOL, Rand, check, ordered, same, sum_tol
from gpu_util import announce, host, torch
from oracle import block as ob

pytestmark = pytest.mark.gpu

# r comes from a float32 sum of G squares, all positive: its relative error is below the number
# of roundings on a term's way (at most 64) times 2^-24, halved by the square root. rstd is
# compared relative to itself.
RSTD_TOL = 64 * 2.0 ** -24



def grad_tol(io, v, shape, mode):
    """dv = r (A - n mean(A n)), n the normed values, is a difference: each of its two terms is
    within 32 roundings (the gate's 8, the products' 4, the mean's sum 20) of 2^-24 of its own
    size, r |A| and r |n| |mean(A n)| <= r |n| rms(A), however small the difference is. In a
    group of one channel n^2 = 1 - eps r^2 and the terms cancel down to eps r^2 of themselves.
    So the bar grows by 32 * 2^-24 times the terms' rms over the difference's (dz, the
    difference times y silu', likewise)."""
    y, w, g = v["y"][1], v["weight"][1], v["dout"][1]
    z = None if mode == "none" else v["z"][1]
    opt = options(shape, mode)
    b, d, L = y.shape
    per = d // shape[3]
    gate = np.ones_like(y) if z is None else z * ob.sigmoid(z)
    A = g * w[None, :, None] * (gate if opt["norm_before_gate"] else 1.0)
    n, rstd = ob.norm_ref(y, np.ones(d), None if opt["norm_before_gate"] else z, 1e-5, shape[3])
    r = np.repeat(rstd, per, axis=1)
    rms_a = np.repeat(np.sqrt((A * A).reshape(b, shape[3], per, L).mean(2)), per, axis=1)
    terms = r * (np.abs(A) + np.abs(n) * rms_a)
    diff = r * (A - n * np.repeat((A * n).reshape(b, shape[3], per, L).mean(2), per, axis=1))
    ratio = np.sqrt((terms ** 2).mean() / (diff ** 2).mean())
    return TOL[io] + 32 * 2.0 ** -24 * ratio


SHAPES = [
    # (batch, dim, seqlen, groups)
    (1, 1, 1, 1), (2, 3, 5, 1), (3, 64, 1, 1), (2, 64, 8, 4), (1, 72, 9, 1), (2, 130, 33, 2),
    (1, 515, 70, 1), (2, 512, 64, 8), (1, 2048, 20, 1), (1, 16, 777, 1), (2, 40, 300, 5),
    (1, 6000, 11, 1), (1, 8200, 9, 1), (1, 16400, 3, 1), (65, 96, 1, 1), (300, 24, 1, 3),
]
ids = lambda s: "b{}d{}L{}g{}".format(*s)
MODES = ["none", "gate_first", "norm_first"]


def make(shape, io, seed):
    b, d, L, _ = shape
    r = Rand(seed)
    return {"y": r((b, d, L), io), "z": r((b, d, L), io), "weight": r((d,)),
            "dout": r((b, d, L), io)}


def options(shape, mode):
    return dict(groups=shape[3], norm_before_gate=mode == "norm_first")


def forward(v, shape, mode, orders, token):
    return ssm.norm_train(ordered(v["y"][0], orders[0]), v["weight"][0],
                          z=None if mode == "none" else ordered(v["z"][0], orders[1]),
                          token_major=token, **options(shape, mode))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_norm_shapes(shape, mode, io):
    for orders, token in ((("time", "channel"), True), (("channel", "odd"), True)):
        announce(f"norm {ids(shape)} {mode} {io} {orders} token {token}")
        v = make(shape, io, 600 + sum(shape))
        out, rstd = forward(v, shape, mode, orders, token)
        ref, rref = ob.norm_ref(v["y"][1], v["weight"][1], None if mode == "none" else v["z"][1],
                                1e-5, **options(shape, mode))
        check(out, ref.transpose(0, 2, 1) if token else ref, TOL[io], "out")
        assert np.abs(host(rstd) / rref - 1).max() <= RSTD_TOL
        # the gradients, from this rstd
        g = ssm.norm_backward(ordered(v["y"][0], orders[0]), v["weight"][0], rstd,
                              (v["dout"][0].transpose(1, 2) if token else v["dout"][0]),
                              z=None if mode == "none" else ordered(v["z"][0], orders[1]),
                              token_major=token, **options(shape, mode))
        gref = ob.norm_bwd_ref(v["y"][1], v["weight"][1], v["dout"][1],
                               None if mode == "none" else v["z"][1], 1e-5,
                               **options(shape, mode))
        check(g["dy"], gref["dy"], grad_tol(io, v, shape, mode), "dy")
        if mode == "none":
            assert g["dz"] is None
        else:
            check(g["dz"], gref["dz"], grad_tol(io, v, shape, mode), "dz")
        check(g["dweight"], gref["dweight"], sum_tol(shape[0] * shape[2]), "dweight")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("z_order", ["time", "channel", "odd"])
@pytest.mark.parametrize("y_order", ["time", "channel", "odd"])
def test_norm_orders(y_order, z_order, token, io):
    """Every order of the inputs and the output gives the same values, and the gradients come
    in their inputs' orders."""
    shape = (2, 136, 50, 2)
    announce(f"norm orders {y_order} {z_order} token {token} {io}")
    v = make(shape, io, 640)
    out, rstd = forward(v, shape, "gate_first", (y_order, z_order), token)
    ref, _ = ob.norm_ref(v["y"][1], v["weight"][1], v["z"][1], 1e-5, 2)
    assert out.is_contiguous()
    check(out, ref.transpose(0, 2, 1) if token else ref, TOL[io], "out")
    dout = v["dout"][0].transpose(1, 2).contiguous() if token else v["dout"][0]
    g = ssm.norm_backward(ordered(v["y"][0], y_order), v["weight"][0], rstd, dout,
                          z=ordered(v["z"][0], z_order), groups=2, token_major=token)
    gref = ob.norm_bwd_ref(v["y"][1], v["weight"][1], v["dout"][1], v["z"][1], 1e-5, 2)
    check(g["dy"], gref["dy"], TOL[io], "dy")
    check(g["dz"], gref["dz"], TOL[io], "dz")
    check(g["dweight"], gref["dweight"], sum_tol(100), "dweight")
    assert g["dy"].stride(2 if y_order == "time" else 1) == 1
    assert g["dz"].stride(2 if z_order == "time" else 1) == 1


@pytest.mark.parametrize("mode", MODES)
def test_norm_rows_of_zeros_and_magnitudes(mode):
    """A token whose values are all zero is 0 / sqrt(eps); tokens of 1e4 and 1e-4 keep their
    relative accuracy; a NaN stays in its token."""
    announce(f"norm magnitudes {mode}")
    t = torch()
    shape = (1, 200, 40, 1)
    v = make(shape, "f32", 650)
    y = v["y"][0]
    y[0, :, 3] = 0
    y[0, :, 5] *= 1e4
    y[0, :, 7] *= 1e-4
    z = None if mode == "none" else v["z"][0]
    first = mode == "norm_first"
    ref, rref = ob.norm_ref(host(y), v["weight"][1], None if z is None else v["z"][1], 1e-5, 1, first)
    out, rstd = ssm.norm_train(y, v["weight"][0], z=z, norm_before_gate=first)
    check(out, ref, TOL["f32"], "out")
    assert np.abs(host(rstd) / rref - 1).max() <= RSTD_TOL
    assert not out[0, :, 3].any()
    g = ssm.norm_backward(y, v["weight"][0], rstd, v["dout"][0], z=z, norm_before_gate=first)
    gref = ob.norm_bwd_ref(host(y), v["weight"][1], v["dout"][1], None if z is None else v["z"][1],
                           1e-5, 1, first)
    for at in (3, 5, 7, 9):  # each token on its own scale
        check(host(g["dy"])[:, :, at], gref["dy"][:, :, at], TOL["f32"], f"dy token {at}")
    y[0, 11, 20] = float("nan")
    bad = t.isnan(ssm.norm(y, v["weight"][0], z=z, norm_before_gate=first))
    want = t.zeros_like(bad)
    want[0, :, 20] = True
    assert t.equal(bad, want)


def test_norm_layer_size():
    """The norm after the Mamba-2 layer's scan (b4, 2048 channels, 2048 steps): the scan's order
    in, a projection's gate, a projection's order out; sampled tokens against the oracle, and
    bitwise reproducible."""
    announce("norm layer")
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(9)
    mk = lambda: t.randn(4, 2048, 2048, device="cuda", generator=gen).bfloat16()
    y, z, dout = mk(), ordered(mk(), "channel"), mk().transpose(1, 2).contiguous()
    w = t.randn(2048, device="cuda", generator=gen)
    out, rstd = ssm.norm_train(y, w, z=z, token_major=True)
    g = ssm.norm_backward(y, w, rstd, dout, z=z, token_major=True)
    at = [0, 1, 7, 8, 31, 32, 1000, 2047]
    pick = lambda v: host(v[:, :, at].contiguous())
    ref, rref = ob.norm_ref(pick(y), host(w), pick(z))
    check(host(out[:, at]), ref.transpose(0, 2, 1), TOL["bf16"], "out")
    gref = ob.norm_bwd_ref(pick(y), host(w), host(dout[:, at]).transpose(0, 2, 1), pick(z))
    check(pick(g["dy"]), gref["dy"], TOL["bf16"], "dy")
    check(pick(g["dz"]), gref["dz"], TOL["bf16"], "dz")
    yd, zd = y.double(), z.double()
    n = yd * zd * t.sigmoid(zd)
    dw = (n * t.rsqrt((n * n).mean(1, keepdim=True) + 1e-5) * dout.double().transpose(1, 2)).sum((0, 2))
    check(g["dweight"], dw.cpu().numpy(), sum_tol(4 * 2048), "dweight")
    again = ssm.norm_backward(y, w, rstd, dout, z=z, token_major=True)
    assert all(same(g[k].contiguous(), again[k].contiguous()) for k in g)


def test_gated_norm_autograd():
    announce("gated_norm autograd")
    for mode in MODES:
        shape = (2, 48, 30, 3)
        v = make(shape, "f32", 660)
        leaf = {k: v[k][0].clone().requires_grad_() for k in ("y", "weight", "z")}
        z = None if mode == "none" else leaf["z"]
        out = ssm.gated_norm(leaf["y"], leaf["weight"], z=z, token_major=True,
                             **options(shape, mode))
        (out * v["dout"][0].transpose(1, 2)).sum().backward()
        ref = ob.norm_bwd_ref(v["y"][1], v["weight"][1], v["dout"][1],
                              None if z is None else v["z"][1], 1e-5, **options(shape, mode))
        for name, key in (("y", "dy"), ("weight", "dweight"), ("z", "dz")):
            if name != "z" or z is not None:
                check(leaf[name].grad, ref[key], sum_tol(60), f"{mode} {key}")


def test_norm_empty():
    announce("norm empty")
    t = torch()
    w = t.ones(6, device="cuda")
    y = t.empty(2, 6, 0, device="cuda")
    out, rstd = ssm.norm_train(y, w, groups=2, token_major=True)
    assert out.shape == (2, 0, 6) and rstd.shape == (2, 2, 0)
    g = ssm.norm_backward(y, w, rstd, out, groups=2, token_major=True)
    assert g["dy"].shape == (2, 6, 0) and not g["dweight"].any()
