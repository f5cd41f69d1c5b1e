"""Shared by the tests of the operators around the scan: inputs in the storage type with their
float64 values, tensors in either memory order, and the comparison."""
import numpy as np

from gpu_util import host, torch
from ssm_workloads import WATCH, parity

# Results computed in float32 and stored in the storage type. bf16: half a step of the rounding,
# 2^-8, and the float32 part (WATCH). float32: sums of at most a few dozen products with one
# rounding each, 2^-24 of the terms' absolute sum, which is below 16 times the scale of the
# metric here (|r| + rms), and a sigmoid whose exponent's rounding adds |p| 2^-24: under
# 64 * 16 * 2^-24 = 6.1e-5.
TOL = {"f32": 6.1e-5, "bf16": WATCH["bf16"]}


def sum_tol(n):
    """A float32 sum of n random terms, compared on the metric |r| + rms: at most 32 roundings
    lie between a term and the result (8 in a lane, 6 across lanes, and the partial sums), each
    2^-24 of an absolute sum that is about sqrt(n) times the rms of the signed one; and the
    terms' own error."""
    return 32 * 2.0 ** -24 * max(n, 1) ** 0.5 + TOL["f32"]


def dtype(io):
    t = torch()
    return t.bfloat16 if io == "bf16" else t.float32


class Rand:
    """Seeded inputs: (device tensor in the storage type, its values as float64)."""

    def __init__(self, seed):
        self.g = torch().Generator().manual_seed(seed)

    def __call__(self, shape, io="f32", scale=1.0, device="cuda"):
        t = torch()
        v = (t.randn(shape, generator=self.g) * scale).to(dtype(io))
        return v.to(device), v.double().numpy()


def ordered(x, order):
    """The [batch, dim, seqlen] tensor x in a memory order: "time" (contiguous), "channel" (a
    slice of a token-major buffer, rows 16-byte aligned where the element size allows) or
    "odd" (the same at an odd offset of an odd row)."""
    t = torch()
    if order == "time":
        return x.contiguous()
    b, d, L = x.shape
    pad, off = (16, 8) if order == "channel" else (13, 5)
    wide = t.full((b, L, d + pad), float("nan"), device=x.device, dtype=x.dtype)
    view = wide[:, :, off:off + d].transpose(1, 2)
    view.copy_(x)
    return view


def check(got, ref, tol, label):
    g = host(got) if not isinstance(got, np.ndarray) else got
    r = parity(g, ref, tol, tol)
    print(f"[parity] {label}: {r}", flush=True)
    assert r.ok, f"{label}: {r}"


def same(a, b):
    t = torch()
    return bool(t.equal(a.view(t.int16) if a.dtype == t.bfloat16 else a.view(t.int32),
                        b.view(t.int16) if b.dtype == t.bfloat16 else b.view(t.int32)))
