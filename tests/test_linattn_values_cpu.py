"""Values that are not finite in linear attention, the kernels in a CPU build: they reach what the recurrence
takes them to, and no step before them."""
import numpy as np
import pytest

from linattn_emulated import CLANG, kernels_of, rounded
from linattn_values import BAD, check_backward, check_forward
from test_linattn_cpu import LARGE

pytestmark = pytest.mark.skipif(CLANG is None, reason="clang++ not available")


@pytest.fixture(scope="module", params=[{}, LARGE], ids=["small", "large"])
def kernels(request):
    return kernels_of(request.param)


def inputs(io, L, hk, h, dk, dv, seed):
    rng = np.random.default_rng(seed)
    draw = lambda *s: rounded(rng.standard_normal(s), io)
    state = lambda: rounded(rng.standard_normal((1, h, dv, dk)), "f32")
    args = dict(q=draw(1, L, hk, dk), k=draw(1, L, hk, dk), v=draw(1, L, h, dv),
                g=rounded(-0.1 * rng.random((1, L, h)), "f32"), initial_state=state())
    return args, draw(1, L, h, dv), state()


PLACES = [("v", (0, 45, 1, 5)), ("v", (0, 64, 0, 17)), ("v", (0, 0, 1, 0)), ("v", (0, 89, 0, 35)),
          ("k", (0, 45, 0, 3)), ("q", (0, 45, 0, 19)), ("g", (0, 50, 1)), ("initial_state", (0, 1, 7, 9))]


# (-inf in g is a reset.)
CASES = [(what, index, bad) for what, index in PLACES for bad in BAD if (what, bad) != ("g", "-inf")]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("what,index,bad", CASES)
def test_forward(kernels, io, what, index, bad):
    args, _, _ = inputs(io, 90, 1, 2, 20, 36, 3)
    check_forward(lambda **a: kernels.forward(io, **a), io, args, what, index, BAD[bad])


GRADIENT_PLACES = PLACES[:6] + [("k", (0, 64, 0, 0)), ("q", (0, 20, 0, 8)), ("dout", (0, 45, 1, 5)), ("dout", (0, 63, 0, 35)),
                                ("initial_state", (0, 1, 7, 9)), ("dfinal", (0, 0, 3, 4))]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("what,index", GRADIENT_PLACES)
def test_gradients(kernels, io, what, index, bad):
    args, dout, dfinal = inputs(io, 90, 1, 2, 20, 36, 4)
    check_backward(lambda **a: kernels.backward(io, **a), io, args, dout, dfinal, what, index, BAD[bad])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("what,index", [("k", (0, 20, 0, 3)), ("dout", (0, 40, 0, 100)), ("q", (0, 50, 0, 1)),
                                        ("v", (0, 9, 1, 64))])
def test_gradients_of_large_heads(kernels, io, what, index):
    args, dout, dfinal = inputs(io, 66, 1, 2, 72, 130, 5)
    check_backward(lambda **a: kernels.backward(io, **a), io, args, dout, dfinal, what, index, np.nan)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("index", [(0, 0, 0), (0, 33, 1), (0, 50, 1), (0, 63, 0), (0, 64, 1), (0, 89, 0)])
def test_gradients_of_decays(kernels, io, bad, index):
    """A decay that is not finite is in dq from its step on, in dk and dv before it, in every dg of its head and in
    dinitial, but in no dk and dv from its step on and in no dq before."""
    args, dout, dfinal = inputs(io, 90, 1, 2, 20, 36, 6)
    args["g"][0, 70, index[2]] = -np.inf  # a reset after or before it does not hide it
    check_backward(lambda **a: kernels.backward(io, **a), io, args, dout, dfinal, "g", index, BAD[bad])
    check_forward(lambda **a: kernels.forward(io, **a), io, args, "g", index, BAD[bad])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("what,index", [("v", (0, 40, 1, 5)), ("k", (0, 40, 0, 3)), ("q", (0, 56, 0, 19)), ("dout", (0, 33, 1, 5)),
                                        ("g", (0, 50, 1)), ("dfinal", (0, 0, 3, 4))])
def test_before_the_end_of_a_row(kernels, io, what, index):
    """A row of 57 of 90 steps, what lies behind its end NaN: only the value before the end is in the results."""
    args, dout, dfinal = inputs(io, 90, 1, 2, 20, 36, 7)
    for x in (args["q"], args["k"], args["v"], args["g"], dout):
        x[:, 57:] = np.nan
    check_backward(lambda **a: kernels.backward(io, **a), io, args, dout, dfinal, what, index, np.nan, [57])
    if what in args:
        check_forward(lambda **a: kernels.forward(io, **a), io, args, what, index, np.nan, [57])
