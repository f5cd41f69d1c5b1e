"""The gated norm's gradient at the ends of float32's range, against the float64 oracle: tokens
whose values, and so whose r = 1 / sqrt(mean + eps), are many powers of ten from one.

The forward is right as long as a token's mean square is a normal float32 number (values of about
1e-18 to 1e18), and its gradient has to be right as far.
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import TOL, Rand, check, dtype, ordered
from gpu_util import announce, host
from oracle import block as ob

pytestmark = pytest.mark.gpu

# By eps: eps 0 leaves tokens of small values as the oracle's 1 / sqrt(mean) takes them.
SCALES = {1e-5: [1.0, 1e3, 1e8, 1e12, 1e14, 1e15, 1e16, 1e17],
          0.0: [1.0, 1e-4, 1e-8, 1e-11, 1e-13, 1e-14, 1e-16, 1e-17]}
MODES = ["none", "gate_first", "norm_first"]


def bar(io, terms, diff):
    """dv = r (A - n mean(A n)) of one token: each of its two terms is within 48 roundings (the
    gate's 8, the products' 8, and 32 in the mean's sum: 8 in a lane, 6 across lanes, 16 waves or
    blocks) of 2^-24 of its own size; the difference may be smaller than they are."""
    ratio = np.sqrt((terms ** 2).mean() / (diff ** 2).mean())
    return TOL[io] + 48 * 2.0 ** -24 * ratio


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("dims", [(200, "time"), (64, "channel"), (6000, "time")],
                         ids=lambda s: f"d{s[0]}-{s[1]}")
def test_norm_gradient_over_the_range(dims, eps, mode, io):
    d, order = dims
    announce(f"norm range d{d} {order} eps {eps} {mode} {io}")
    scales = SCALES[eps]
    L = len(scales)
    r = Rand(700 + d)
    y = (r((1, d, L))[0] * r((1, 1, L))[0].new_tensor(scales)).to(dtype(io))
    (z, z64), (g, g64), (w, w64) = r((1, d, L), io), r((1, d, L), io), r((d,))
    y64 = host(y)
    first, gated = mode == "norm_first", mode != "none"
    opt = dict(z=ordered(z, "channel") if gated else None, norm_before_gate=first)
    out, rstd = ssm.norm_train(ordered(y, order), w, eps=eps, **opt)
    ref, rref = ob.norm_ref(y64, w64, z64 if gated else None, eps, 1, first)
    got = ssm.norm_backward(ordered(y, order), w, rstd, g, **opt)
    gref = ob.norm_bwd_ref(y64, w64, g64, z64 if gated else None, eps, 1, first)
    gate = z64 * ob.sigmoid(z64) if gated else np.ones_like(y64)
    A = g64 * w64[None, :, None] * (gate if first else 1.0)
    n = (y64 if first else y64 * gate) * rref
    m = (A * n).mean(1, keepdims=True)
    rms = np.sqrt((A * A).mean(1, keepdims=True))
    terms, diff = rref * (np.abs(A) + np.abs(n) * rms), rref * (A - n * m)
    for t, scale in enumerate(scales):  # each token on its own scale
        at = lambda v: v[:, :, t]
        check(at(host(out)), at(ref), TOL[io], f"out at {scale}")
        tol = bar(io, at(terms), at(diff))
        check(at(host(got["dy"])), at(gref["dy"]), tol, f"dy at {scale}")
        if gated:
            check(at(host(got["dz"])), at(gref["dz"]), tol, f"dz at {scale}")
    check(got["dweight"], gref["dweight"], 48 * 2.0 ** -24 * L ** 0.5 + TOL["f32"], "dweight")
