"""Views of the imaginary part of a conjugate, whose memory holds the negative of their values, as
inputs of the operators around the scan: the values count. Both ways of marshalling a call."""
import pytest

import selective_state_space_fwd_amd as ssm
from gpu_util import announce, torch
from selective_state_space_fwd_amd import block

pytestmark = pytest.mark.gpu


def negative(v):
    """(a view whose memory holds -v, v): with one step or row it passes for contiguous."""
    t = torch()
    view = t.complex(t.zeros_like(v), -v).conj().imag
    assert view.is_neg() and t.equal(view, v)
    return view


@pytest.mark.parametrize("native", [True, False])
def test_negative_views(native, monkeypatch):
    announce(f"negative views, module {native}")
    t = torch()
    block._load()
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    g = t.Generator().manual_seed(6)
    mk = lambda *s: t.randn(s, generator=g).cuda()
    for b, d, L in ((2, 6, 1), (1, 1, 1), (1, 1, 5), (2, 6, 5)):
        x, w, dout, n = mk(b, d, L), mk(d, 4), mk(b, d, L), mk(d)
        row, A, B, st, cs = mk(b, d), -mk(d, 1).abs(), mk(b, 1), mk(b, d, 1), mk(b, d, 3)
        rstd = ssm.norm_train(x, n, z=dout)[1]

        def calls(f):
            s1, s2, s3 = cs.clone(), st.clone(), st.clone()
            got = [*ssm.conv(f(x), w, initial_state=f(cs)), ssm.conv(x, f(w), bias=f(n))[0],
                   ssm.conv_step(f(row), s1, w), s1, ssm.scan_step(f(row), f(row), f(A), f(B), f(B), s2, z=f(row)), s2,
                   ssm.ssd_step(row, f(row[:, :1].contiguous()), f(A[:1, 0].contiguous()), B, B, s3, D=f(n)), s3,
                   ssm.norm(f(x), n, z=f(dout), token_major=True), ssm.norm(x, f(n))]
            for grads in (ssm.conv_backward(f(x), w, f(dout)), ssm.norm_backward(f(x), n, rstd, f(dout), z=f(x))):
                got += [v for v in grads.values() if v is not None]
            return got
        for i, (a, c) in enumerate(zip(calls(lambda v: v), calls(negative))):
            assert t.equal(a, c), (b, d, L, i)


@pytest.mark.parametrize("native", [True, False])
def test_negative_views_are_not_written(native, monkeypatch):
    announce(f"negative results, module {native}")
    t = torch()
    block._load()
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    one = lambda *s: t.ones(s, device="cuda")
    for call in (lambda: ssm.conv(one(1, 1, 1), one(1, 4), out=negative(one(1, 1, 1))),
                 lambda: ssm.conv_step(one(1, 1), negative(one(1, 1, 1)), one(1, 2)),
                 lambda: ssm.scan_step(one(1, 1), one(1, 1), one(1, 1), one(1, 1), one(1, 1), negative(one(1, 1, 1))),
                 lambda: ssm.norm(one(1, 1, 1), one(1), out=negative(one(1, 1, 1)))):
        with pytest.raises(ValueError):
            call()
