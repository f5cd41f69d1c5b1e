"""GPU parity of the queries' and keys' norm and rotation (qk_norm and its gradient) against the float64
oracle (oracle/linattn.py).

Bounds, element by element: everything is float32 but the storage type, a mean of at most 256 squares
and one root and division (under 300 roundings of 2^-24 in the norm, halved by the root), a product
with the weight and two with the angles: a result is off by its own rounding and by under 400 * 2^-24
of its terms, |a| + |b| of a turned pair. dx = r (u - n mean(u n)) is a difference, which may leave
nothing of its terms (a head of one value has a gradient of eps / x^2 times them), so that its error
is measured by them too: with u in absolute terms, 800 * 2^-24 of r (u + |n| mean(u |n|)). The
weights' gradients are sums of n such terms, on the metric |r| + rms of the comparison.
"""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import TOL, Rand, check, same, sum_tol
from linattn_util import U
from gpu_util import announce, host, torch
from oracle import linattn as ol

pytestmark = pytest.mark.gpu

# batch, steps, q heads, k heads, dim, rot, interleaved, positions, weights
SHAPES = [
    (1, 1, 1, 1, 2, 2, False, False, True), (1, 1, 1, 1, 1, 0, False, False, False),
    (2, 9, 4, 2, 128, 128, False, True, True), (3, 50, 5, 5, 96, 48, True, False, True),
    (1, 33, 8, 1, 64, 64, False, True, True), (2, 17, 3, 2, 33, 10, False, True, False),
    (2, 17, 2, 3, 33, 32, True, True, True), (1, 300, 16, 16, 256, 256, False, False, True),
    (4, 2, 2, 1, 256, 2, True, True, True), (2, 5, 3, 3, 80, 0, False, False, True),
    (1, 7, 2, 2, 250, 90, False, True, True), (2, 700, 32, 8, 64, 32, False, True, True),
    (2, 3, 0, 2, 64, 64, False, False, True), (2, 3, 2, 0, 64, 64, True, False, True),
]


def make(shape, io, seed=3, offset=5):
    b, L, hq, hk, d, rot, inter, places, weights = shape
    t, r = torch(), Rand(seed)
    wide, wide64 = r((b, L, (hq + hk) * d + offset), io)
    view = lambda x, at, n: x[..., at:at + n * d].unflatten(-1, (n, d))
    cut = lambda x, at, n: x[..., at:at + n * d].reshape(b, L, n, d)
    q, k = view(wide, offset, hq), view(wide, offset + hq * d, hk)
    q64, k64 = cut(wide64, offset, hq), cut(wide64, offset + hq * d, hk)
    qw, kw = (r((d,)), r((d,))) if weights else ((None, None), (None, None))
    rng = np.random.default_rng(seed)
    rows, opt, ref = 3 * L, {}, {}
    if rot:
        angle = rng.standard_normal((rows, rot // 2)) * 3
        ref = dict(cos=np.cos(angle).astype(np.float32), sin=np.sin(angle).astype(np.float32))
        opt = {n: t.from_numpy(x).cuda() for n, x in ref.items()}
        if places:
            pos = rng.integers(-2, rows + 2, (b, L)).astype(np.int32)
            ref["positions"], opt["positions"] = pos, t.from_numpy(pos).cuda()
    ref["interleaved"] = opt["interleaved"] = inter
    return (q, k), (q64, k64), (qw, kw), opt, ref, r


def pairs(x, rot, interleaved):
    """|a| + |b| in the places of each turned pair, |x| elsewhere."""
    y = np.abs(x)
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + (1 if interleaved else rot // 2)
    y[..., i] = y[..., j] = y[..., i] + y[..., j]
    return y


def close(got, ref, terms, roundings, io, label):
    tol = U[io] * np.abs(ref) + roundings * 2.0 ** -24 * terms + 1e-37
    ratio = float((np.abs(host(got) - ref) / tol).max()) if ref.size else 0.0
    print(f"[bound] {label}: {ratio:.3f} of the bound", flush=True)
    assert ratio <= 1, (label, ratio)


def check_side(name, x64, w, g64, out, d, ref, rot, io, eps=1e-6):
    inter = ref["interleaved"]
    r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
    n, wide = np.abs(x64 * r), 1.0 if w[1] is None else np.abs(w[1])
    close(out, ol.qk_norm_ref(x64, w[1], **ref), pairs(n * wide, rot, inter), 400, io, name)
    dx, dw = ol.qk_norm_bwd_ref(x64, g64, w[1], **ref)
    u = pairs(g64, rot, inter) * wide
    close(d["d" + name], dx, r * (u + n * (u * n).mean(-1, keepdims=True)), 800, io, "d" + name)
    if w[0] is None:
        assert d[f"d{name}_weight"] is None
    else:
        check(d[f"d{name}_weight"], dw, sum_tol(x64[..., 0].size), name + " weight")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["b{}L{}q{}k{}d{}r{}".format(*s[:6]) for s in SHAPES])
def test_qk(shape, io):
    announce(f"qk_norm {shape} {io}")
    (q, k), (q64, k64), (qw, kw), opt, ref, r = make(shape, io)
    out = ssm.qk_norm(q, k, qw[0], kw[0], **opt)
    (gq, gq64), (gk, gk64) = r(q.shape, io), r(k.shape, io)
    d = ssm.qk_norm_backward(q, k, gq, gk, qw[0], kw[0], **opt)
    check_side("q", q64, qw, gq64, out[0], d, ref, shape[5], io)
    check_side("k", k64, kw, gk64, out[1], d, ref, shape[5], io)


# Calls of many heads, whose counts leave the last of a group's heads and the last round of items short.
LARGE = [
    (3, 1501, 7, 3, 96, 48, True, True, True), (2, 6503, 5, 2, 33, 10, False, True, True),
    (1, 2050, 9, 2, 256, 256, False, False, True), (2, 2049, 13, 1, 128, 64, False, True, False),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", LARGE, ids=["b{}L{}q{}k{}d{}r{}".format(*s[:6]) for s in LARGE])
def test_qk_large(shape, io):
    test_qk(shape, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strides(io):
    announce(f"qk_norm strides {io}")
    shape = (2, 40, 4, 2, 64, 64, False, True, True)
    (q, k), _, (qw, kw), opt, _, r = make(shape, io)
    (gq, _), (gk, _) = r(q.shape, io), r(k.shape, io)
    want = ssm.qk_norm(q.contiguous(), k.contiguous(), qw[0], kw[0], **opt)
    grads = ssm.qk_norm_backward(q.contiguous(), k.contiguous(), gq, gk, qw[0], kw[0], **opt)
    major = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)
    last = lambda x: x.transpose(2, 3).contiguous().transpose(2, 3)
    for form in (lambda x: x, major, last):
        got = ssm.qk_norm(form(q), form(k), qw[0], kw[0], **opt)
        assert all(same(x, y) for x, y in zip(got, want))
        d = ssm.qk_norm_backward(form(q), form(k), form(gq), form(gk), qw[0], kw[0], **opt)
        assert all(same(d[n], grads[n]) for n in grads)
    out = [torch().empty_like(x) for x in want]
    again = ssm.qk_norm(q, k, qw[0], kw[0], q_out=out[0], k_out=out[1], **opt)
    assert again[0] is out[0] and again[1] is out[1] and same(out[0], want[0])


def test_ranges():
    """Values of 1e-15 and 1e15, rows of zeros, and a NaN or infinity, which stays in its head."""
    t = torch()
    announce("qk_norm ranges")
    x = t.randn(2, 8, 4, 64, device="cuda")
    scale = t.logspace(-15, 15, 16, device="cuda").reshape(2, 8, 1, 1)
    x64 = host(x * scale)
    out, _ = ssm.qk_norm(x * scale, x, eps=0.0)
    check(out, ol.qk_norm_ref(x64, eps=0.0), TOL["f32"], "ranges")
    zero, _ = ssm.qk_norm(t.zeros_like(x), x)
    assert (zero == 0).all()
    clean, _ = ssm.qk_norm(x, x)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[1, 3, 2, 5] = bad
        out, _ = ssm.qk_norm(y, x)
        assert out[1, 3, 2].isnan().any()
        out[1, 3, 2] = clean[1, 3, 2]
        assert same(out, clean)


def test_empty():
    t = torch()
    announce("qk_norm empty")
    for b, L in ((0, 4), (3, 0)):
        q, w = t.zeros(b, L, 2, 16, device="cuda"), t.ones(16, device="cuda")
        assert all(o.shape == q.shape for o in ssm.qk_norm(q, q, w, w))
        d = ssm.qk_norm_backward(q, q, q, q, w, w)
        assert (d["dq_weight"] == 0).all() and (d["dk_weight"] == 0).all()


def test_many_rows():
    """Rows past 2^31 elements, the last against the same alone."""
    t = torch()
    announce("qk_norm many rows")
    q = t.empty(2, 1 << 17, 72, 128, device="cuda", dtype=t.bfloat16)
    q.view(-1).view(t.int16).fill_(0x3f80)
    q[1, -1] = t.randn(72, 128, device="cuda").bfloat16()
    k, w = q[:, :, :1], t.rand(128, device="cuda")
    out, ko = ssm.qk_norm(q, k, w, w)
    want, kw = ssm.qk_norm(q[1:, -1:], k[1:, -1:], w, w)
    assert same(out[1:, -1:], want) and same(ko[1:, -1:], kw) and same(out[0, 0], out[1, 5])
