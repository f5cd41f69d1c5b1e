"""Gradients of log decays next to much stronger ones on the device: each within the bound of its own
terms, and exactly 0 at a reset."""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from gpu_util import announce, host
from linattn_util import Attention, within
from oracle import linattn as ol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128), (33, 20), (256, 130)])
@pytest.mark.parametrize("L", [150, 700])
def test_dg_of_strong_decays(L, dk, dv, io):
    """(700 steps of one head pair are cut into segments or joined, 150 walked or joined in one.)"""
    announce(f"linattn dg of strong decays L{L} {dk}x{dv} {io}")
    a = Attention(1, L, 1, 2, dk, dv, io, "token", None, True, seed=61, rate=0.02)
    every = np.random.default_rng(62)
    for t in range(3, L, 9):
        a.g[:, t, 0] = -float(every.uniform(4, 60))
        a.g[:, t, 1] = float("-inf") if t % 2 else -20.0
    a.g64 = host(a.g)
    got = ssm.linattn_backward(a.q, a.k, a.v, a.dout, dfinal=a.ds, **a.args())["dg"]
    ref = ol.linattn_bwd_ref(a.q64, a.k64, a.v64, a.dout64, dfinal=a.ds64, **a.ref_args())["dg"]
    ab = ol.linattn_bwd_ref(*map(np.abs, (a.q64, a.k64, a.v64, a.dout64)), dfinal=np.abs(a.ds64), **a.abs_args())["dg"]
    within(got, ref, ab, "f32", 2 * a.roundings, "dg")
    assert (host(got)[np.isinf(a.g64)] == 0).all()
