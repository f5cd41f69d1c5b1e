"""Gradients of log decays where some are much stronger than their neighbours, from the kernels in a CPU
build: each within the bound of its own terms, and exactly 0 at a reset."""
import numpy as np
import pytest

from linattn_emulated import CLANG, kernels_of, rounded
from linattn_util import roundings
from oracle import linattn as ol
from test_linattn_cpu import LARGE

pytestmark = pytest.mark.skipif(CLANG is None, reason="clang++ not available")


@pytest.fixture(scope="module", params=[{}, LARGE], ids=["small", "large"])
def kernels(request):
    return kernels_of(request.param)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,hk", [(64, 64, 1), (20, 36, 1), (128, 130, 2)])
def test_dg_of_strong_decays(kernels, io, dk, dv, hk):
    """Every value of dg is a sum of terms that its decay scales, all of them added: it is off by the
    float32 roundings of those terms alone (linattn_util.roundings, twice as in the other bounds of dg),
    however large the sums of its chunk are."""
    rng = np.random.default_rng(dk + dv)
    b, L, h = 1, 150, 2
    draw = lambda *s: rounded(rng.standard_normal(s), io)
    q, k, v, do = draw(b, L, hk, dk), draw(b, L, hk, dk), draw(b, L, h, dv), draw(b, L, h, dv)
    s0, ds = (rounded(rng.standard_normal((b, h, dv, dk)), "f32") for _ in range(2))
    g = np.full((b, L, h), -0.01)
    strong = {3: -4.0, 9: -60.0, 31: -20.0, 32: -12.0, 40: -15.0, 47: -30.0, 48: -8.0, 64: -25.0, 100: -40.0, 149: -18.0}
    resets = {20: -np.inf, 63: -np.inf, 80: -3e38, 127: -np.inf}
    for t, x in strong.items():
        g[:, t, 0] = x
    for t, x in {**strong, **resets}.items():
        g[:, t, 1] = x
    g = rounded(g, "f32")
    ref = ol.linattn_bwd_ref(q, k, v, do, g, initial_state=s0, dfinal=ds)["dg"]
    ab = ol.linattn_bwd_ref(*map(np.abs, (q, k, v, do)), g, initial_state=np.abs(s0), dfinal=np.abs(ds))["dg"]
    got = kernels.backward(io, q, k, v, do, g, s0, None, ds)["dg"]
    tol = 2 * roundings(dk, dv, L) * 2.0 ** -24 * ab + 1e-37
    ratio = np.abs(got - ref) / tol
    print("worst", ratio.max(), np.unravel_index(ratio.argmax(), ratio.shape))
    assert (ratio <= 1).all(), [(tuple(i), got[tuple(i)], ref[tuple(i)]) for i in np.argwhere(ratio > 1)[:6]]
    assert all(got[0, t, 1] == 0 for t in resets)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_dg_of_heads(kernels, io):
    """One decay for each head: the sum of the steps', none of them there without its terms."""
    rng = np.random.default_rng(5)
    draw = lambda *s: rounded(rng.standard_normal(s), io)
    b, L, h, dk, dv = 2, 70, 3, 16, 24
    q, k, v, do = draw(b, L, 1, dk), draw(b, L, 1, dk), draw(b, L, h, dv), draw(b, L, h, dv)
    g = rounded([-0.02, -25.0, -1e5], "f32")
    args = dict(lengths=[70, 33])
    ref = ol.linattn_bwd_ref(q, k, v, do, g, **args)["dg"].sum((0, 1))
    ab = ol.linattn_bwd_ref(*map(np.abs, (q, k, v, do)), g, **args)["dg"].sum((0, 1))
    got = kernels.backward(io, q, k, v, do, g, **args)["dg"]
    assert (np.abs(got - ref) <= 2 * roundings(dk, dv, L) * 2.0 ** -24 * ab + 1e-37).all(), (got, ref)
    assert got[2] == 0
