"""Steps of the queries' and keys' norm that are padding (a position below 0), the kernels in a CPU build: zeros
and no gradient, with a rotation and without one."""
import numpy as np
import pytest

from linattn_emulated import CLANG, kernels_of, rounded
from linattn_util import U
from oracle import linattn as ol
from test_linattn_cpu import LARGE

pytestmark = pytest.mark.skipif(CLANG is None, reason="clang++ not available")


@pytest.fixture(scope="module", params=[{}, LARGE], ids=["small", "large"])
def kernels(request):
    return kernels_of(request.param)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rot", [0, 8])
def test_padding(kernels, io, rot):
    rng = np.random.default_rng(rot + 1)
    b, L, hq, hk, d = 2, 7, 3, 2, 24
    draw = lambda *s: rounded(rng.standard_normal(s), io)
    q, k, gq, gk = draw(b, L, hq, d), draw(b, L, hk, d), draw(b, L, hq, d), draw(b, L, hk, d)
    w = rounded(1 + 0.1 * rng.standard_normal(d), "f32")
    pos = np.arange(L) + np.array([[0], [3]])
    pad = np.zeros((b, L), bool)
    pad[0, 4:], pad[1, 0] = True, True
    pos[pad] = [-1, -5, -2 ** 31, -1]
    cos = sin = None
    if rot:
        angle = rng.standard_normal((20, rot // 2))
        cos, sin = rounded(np.cos(angle), "f32"), rounded(np.sin(angle), "f32")
    q[pad], k[pad], gq[pad] = np.nan, np.inf, np.nan
    with np.errstate(all="ignore"):
        got = kernels.qk(io, q, k, w, w, cos, sin, pos, gq, gk)
    for x, g, out, dx, dw in ((q, gq, got[0], got[2], got[4]), (k, gk, got[1], got[3], got[5])):
        assert (out[pad] == 0).all() and (dx[pad] == 0).all()
        x, g = (np.where(pad[:, :, None, None], 0.0, y) for y in (x, g))
        at = np.where(pad, 0, pos)
        want = ol.qk_norm_ref(x, w, cos, sin, positions=at)
        dxw, dww = ol.qk_norm_bwd_ref(x, g, w, cos, sin, positions=at)
        # float32 throughout, a few dozen roundings, and the result's own; a weight's gradient is a sum of 42 terms
        # of a few units at most
        tol = lambda y: U[io] * np.abs(y) + 64 * 2.0 ** -24 * 8
        live = ~pad
        assert (np.abs(out - want)[live] <= tol(want)[live]).all()
        assert (np.abs(dx - dxw)[live] <= tol(dxw)[live]).all()
        assert (np.abs(dw - dww) <= 256 * 2.0 ** -24 * 42).all()
