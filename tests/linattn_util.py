"""Shared by the tests of linear attention and of the queries' and keys' norm: inputs, and bounds on
each element's error.

Every result is a sum of products with positive decays between, so the oracle run on the inputs'
absolute values gives the sum of the absolute values of a result's terms. An element may be off by

  u |result|                      its rounding to the storage type: bf16 2^-8, float32 2^-24
  + p (sum of absolute terms)     the weights of the pairs of a chunk, rounded to bf16 once as operands:
                                  2^-8 in bf16, nothing in float32
  + n 2^-24 (sum of absolute terms)   n float32 roundings on a term's way into the result
"""
import numpy as np

from block_util import Rand, dtype
from gpu_util import host, torch

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
P = {"f32": 0.0, "bf16": 2.0 ** -8}


def roundings(dk, dv, L):
    """float32 roundings between a term and a result, at most: the contractions over a head (dk, dv)
    and over a chunk (64), twice where one result feeds another, one decay factor and one sum a
    chunk, two roundings in each of four decay factors and 32 for their exponents (an exponent's
    rounding is 2^-24 of it, and a decay of exp(-32) leaves nothing to be wrong about), and the
    scale. A state in two bf16 pieces is off by 2^-17, 128 roundings."""
    return 2 * (dk + dv + 2 * 64) + 2 * (L // 32 + 1) + 8 + 32 + 2 + 128


def within(got, ref, absolute, io, n, label, pairs=True):
    g = host(got) if not isinstance(got, np.ndarray) else got
    assert g.shape == ref.shape, (label, g.shape, ref.shape)
    tol = U[io] * np.abs(ref) + ((P[io] if pairs else 0.0) + n * 2.0 ** -24) * absolute + 1e-37
    bad = ~(np.abs(g - ref) <= tol)
    ratio = float(np.max(np.abs(g - ref) / tol)) if g.size else 0.0
    print(f"[bound] {label}: {ratio:.3f} of the bound", flush=True)
    assert not bad.any(), (label, ratio, int(bad.sum()), np.argwhere(bad)[:4].tolist())


class Attention:
    """Inputs of one call on the device (q, k and v slices of one projection) and as float64."""

    def __init__(self, b, L, hk, h, dk, dv, io, decay="token", lengths=None, state=False, seed=0,
                 offset=0, rate=0.3):
        t = torch()
        r = Rand(seed)
        self.io, self.sizes, self.lengths = io, (b, L, hk, h, dk, dv), lengths
        width = 2 * hk * dk + h * dv + offset
        wide, wide64 = r((b, L, width), io)
        if lengths is not None:  # behind a row's length nothing may be read
            for i, n in enumerate(lengths):
                wide[i, max(0, min(n, L)):] = float("nan")
        cut = lambda x, at, n, d: x[..., at:at + n * d].reshape(*x.shape[:2], n, d)
        view = lambda x, at, n, d: x[..., at:at + n * d].unflatten(-1, (n, d))
        at = (offset, offset + hk * dk, offset + 2 * hk * dk)
        self.q, self.k = view(wide, at[0], hk, dk), view(wide, at[1], hk, dk)
        self.v = view(wide, at[2], h, dv)
        self.q64, self.k64 = cut(wide64, at[0], hk, dk), cut(wide64, at[1], hk, dk)
        self.v64 = cut(wide64, at[2], h, dv)
        self.g = self.g64 = None
        if decay != "none":
            x, _ = r((h,) if decay == "head" else (b, L, h))
            self.g = -rate * x.abs()
            self.g64 = host(self.g)
            if lengths is not None and decay == "token":
                for i, n in enumerate(lengths):
                    self.g[i, max(0, min(n, L)):] = float("nan")
        self.s0, self.s064 = r((b, h, dv, dk)) if state else (None, None)
        self.dout, self.dout64 = r((b, L, h, dv), io)
        self.ds, self.ds64 = r((b, h, dv, dk)) if state else (None, None)
        self.n = None if lengths is None else t.tensor(lengths, dtype=t.int32, device="cuda")

    def args(self):
        return dict(g=self.g, initial_state=self.s0, lengths=self.n)

    def ref_args(self):
        return dict(g=self.g64, initial_state=self.s064, lengths=self.lengths)

    def abs_args(self):
        return dict(g=self.g64, initial_state=None if self.s064 is None else np.abs(self.s064),
                    lengths=self.lengths)

    @property
    def roundings(self):
        b, L, hk, h, dk, dv = self.sizes
        return roundings(dk, dv, L)


def reach(absolute, chunk=64):
    """For dg, whose sums within a chunk are differences of running sums: the sum of absolute terms
    over the chunk ([batch, seqlen, heads])."""
    out = np.empty_like(absolute)
    for t in range(0, absolute.shape[1], chunk):
        out[:, t:t + chunk] = absolute[:, t:t + chunk].sum(1, keepdims=True)
    return out
