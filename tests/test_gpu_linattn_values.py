"""Values that are not finite in linear attention on the device: they reach what the recurrence takes them to,
and no step before them. (The forms of the kernels: head sizes, rows by words and by elements, whole sequences and
segments.)"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import dtype
from gpu_util import announce, host, torch
from linattn_values import BAD, check_backward, check_forward

pytestmark = pytest.mark.gpu

# steps, query heads, heads, dk, dv
SHAPES = [(90, 1, 2, 64, 64), (150, 1, 2, 128, 128), (700, 1, 1, 64, 128), (100, 2, 2, 33, 20), (130, 1, 2, 100, 100),
          (70, 1, 1, 256, 130), (140, 1, 4, 128, 64)]
IDS = ["L{}hk{}h{}k{}v{}".format(*s) for s in SHAPES]


def inputs(io, shape, seed):
    """Values that the storage type holds, as float64."""
    t = torch()
    L, hk, h, dk, dv = shape
    gen = t.Generator().manual_seed(seed)
    draw = lambda *s: t.randn(s, generator=gen).to(dtype(io)).double().numpy()
    state = lambda: t.randn(1, h, dv, dk, generator=gen).double().numpy()
    args = dict(q=draw(1, L, hk, dk), k=draw(1, L, hk, dk), v=draw(1, L, h, dv),
                g=-0.1 * t.rand(1, L, h, generator=gen).double().numpy(), initial_state=state())
    return args, draw(1, L, h, dv), state()


def device(x, io="f32"):
    return None if x is None else torch().from_numpy(x).to(dtype(io)).cuda()


def forward(io):
    def call(q, k, v, g, initial_state, lengths=None):
        out, fin = ssm.linattn(device(q, io), device(k, io), device(v, io), device(g), initial_state=device(initial_state))
        return host(out), host(fin)
    return call


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, io):
    args, _, _ = inputs(io, shape, 71)
    rng = np.random.default_rng(72)
    for bad in BAD:
        for what in ("v", "v", "k", "q", "g", "initial_state"):
            if (what, bad) == ("g", "-inf"):  # a reset
                continue
            index = [int(rng.integers(n)) for n in args[what].shape]
            index[1] = max(index[1], 1) if what != "initial_state" else index[1]
            index = tuple(index)
            announce(f"linattn {shape} {io} {bad} in {what} at {index}")
            check_forward(forward(io), io, args, what, index, BAD[bad])


def backward(io):
    def call(q, k, v, dout, g, initial_state, dfinal, lengths=None):
        d = ssm.linattn_backward(device(q, io), device(k, io), device(v, io), device(dout, io), device(g),
                                 initial_state=device(initial_state), dfinal=device(dfinal))
        return {n: host(x) for n, x in d.items()}
    return call


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gradients(shape, io):
    args, dout, dfinal = inputs(io, shape, 74)
    rng = np.random.default_rng(75)
    arrays = dict(args, dout=dout, dfinal=dfinal)
    for bad in BAD:
        for what in ("v", "k", "k", "q", "q", "dout", "dout", "initial_state", "dfinal"):
            index = tuple(int(rng.integers(n)) for n in arrays[what].shape)
            announce(f"linattn_backward {shape} {io} {bad} in {what} at {index}")
            check_backward(backward(io), io, args, dout, dfinal, what, index, BAD[bad])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gradients_of_decays(shape, io):
    args, dout, dfinal = inputs(io, shape, 76)
    rng = np.random.default_rng(77)
    args["g"][0, shape[0] // 2] = -np.inf  # (a reset does not hide it)
    for bad in ("nan", "inf"):
        for _ in range(2):
            index = tuple(int(rng.integers(n)) for n in args["g"].shape)
            announce(f"linattn_backward {shape} {io} {bad} in g at {index}")
            check_backward(backward(io), io, args, dout, dfinal, "g", index, BAD[bad])


def test_uninitialised_padding():
    """A prompt padded behind its end with whatever memory holds, the caller cutting the results: the rows before
    are those of the prompt alone."""
    t = torch()
    announce("linattn padding that is not finite")
    shape = (100, 1, 2, 64, 64)
    for io in ("f32", "bf16"):
        args, _, _ = inputs(io, shape, 73)
        q, k, v = (device(args[n], io) for n in "qkv")
        g = device(args["g"])
        want = ssm.linattn(q[:, :77], k[:, :77], v[:, :77], g[:, :77])[0]
        for x in (q, k, v, g):
            x[:, 77:] = float("nan")
        got = ssm.linattn(q, k, v, g)[0][:, :77]
        assert t.isfinite(got).all()
        tol = 2.0 ** -7 if io == "bf16" else 2.0 ** -20  # two bf16 roundings of a result, and sums in other orders
        assert (got.float() - want.float()).norm() <= tol * want.float().norm()
