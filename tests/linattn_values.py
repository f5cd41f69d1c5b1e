"""Shared by the tests of values that are not finite in linear attention: the recurrence step by step says
which elements of a result they reach, and no other may be anything but its value."""
import numpy as np

from linattn_util import P, U, roundings
from oracle import linattn as ol

BAD = {"nan": np.nan, "inf": np.inf, "-inf": -np.inf}


def only_where(got, ref, absolute, io, n, label, pairs=True):
    """Not finite exactly where the recurrence is not, within the bounds of linattn_util elsewhere
    (absolute: the sums of absolute terms, the bad value 0 among them)."""
    good = np.isfinite(ref)
    assert got.shape == ref.shape, label
    wrong = np.isfinite(got) != good
    assert not wrong.any(), (label, "finite" if np.isfinite(got[wrong][0]) else "not finite", int(wrong.sum()),
                             np.argwhere(wrong)[:6].tolist())
    tol = U[io] * np.abs(ref[good]) + ((P[io] if pairs else 0.0) + n * 2.0 ** -24) * absolute[good] + 1e-37
    assert (np.abs(got[good] - ref[good]) <= tol).all(), label


def place(x, index, bad):
    """x with one bad value, and x with 0 there."""
    with_it, without = x.copy(), x.copy()
    with_it[index] = bad
    without[index] = 0.0
    return with_it, without


def check_forward(call, io, args, what, index, bad, lengths=None):
    """args: q, k, v, g, initial_state as float64; call(q=..., ...) gives (out, final) as float64."""
    dk, dv, L = args["q"].shape[3], args["v"].shape[3], args["q"].shape[1]
    n = roundings(dk, dv, L)
    dirty, clean = dict(args), dict(args)
    dirty[what], clean[what] = place(args[what], index, bad)
    with np.errstate(all="ignore"):
        ref = ol.linattn_ref(**dirty, lengths=lengths)
        ab = ol.linattn_ref(**{k: x if k == "g" or x is None else np.abs(x) for k, x in clean.items()}, lengths=lengths)
        got = call(**dirty, lengths=lengths)
    assert not np.isfinite(ref[0]).all() and np.isfinite(ref[0]).any()
    only_where(got[0], ref[0], ab[0], io, n, f"out, {what} {bad}")
    only_where(got[1], ref[1], ab[1], "f32", n, f"final state, {what} {bad}")


def check_backward(call, io, args, dout, dfinal, what, index, bad, lengths=None):
    """As check_forward; `what` may be dout or dfinal too. call(dout=..., dfinal=..., ...) gives the gradients, dg of
    each step."""
    dk, dv, L = args["q"].shape[3], args["v"].shape[3], args["q"].shape[1]
    n = roundings(dk, dv, L)
    dirty = dict(args, dout=dout, dfinal=dfinal)
    clean = dict(dirty)
    dirty[what], clean[what] = place(dirty[what], index, bad)
    with np.errstate(all="ignore"):
        ref = ol.linattn_bwd_ref(**dirty, lengths=lengths)
        ab = ol.linattn_bwd_ref(**{k: x if k == "g" or x is None else np.abs(x) for k, x in clean.items()},
                                lengths=lengths)
        got = call(**dirty, lengths=lengths)
    assert any(not np.isfinite(x).all() for x in ref.values()) and any(np.isfinite(x).any() for x in ref.values())
    for name in ("dq", "dk", "dv"):
        only_where(got[name], ref[name], ab[name], io, n, f"{name}, {what} {bad}")
    only_where(got["dinitial"], ref["dinitial"], ab["dinitial"], "f32", n, f"dinitial, {what} {bad}")
    only_where(got["dg"], ref["dg"], ab["dg"], "f32", 2 * n, f"dg, {what} {bad}")
