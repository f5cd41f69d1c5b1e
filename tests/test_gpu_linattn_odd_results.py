"""Results of linear attention at addresses of one element's alignment (bf16: 2 bytes): the bits of aligned
ones, and nothing written beside them."""
import ctypes

import pytest

import selective_state_space_fwd_amd as ssm
from block_util import same
from gpu_util import announce, torch
from linattn_util import Attention

pytestmark = pytest.mark.gpu
GUARD = 64


def odd(shape, offset):
    """A contiguous view `offset` elements into a buffer of ones, and the buffer."""
    t = torch()
    n = 1
    for s in shape:
        n *= s
    buf = t.ones(n + 2 * GUARD, dtype=t.bfloat16, device="cuda")
    return buf[GUARD + offset:GUARD + offset + n].view(shape), buf


def untouched(buf, offset, n):
    return bool((buf[:GUARD + offset] == 1).all() and (buf[GUARD + offset + n:] == 1).all())


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 72)])
def test_forward(dk, dv, offset):
    announce(f"linattn out {offset} elements on, {dk}x{dv}")
    a = Attention(1, 100, 1, 2, dk, dv, "bf16", "token", None, True, seed=31)
    want = ssm.linattn(a.q, a.k, a.v, **a.args())
    out, buf = odd((1, 100, 2, dv), offset)
    got = ssm.linattn(a.q, a.k, a.v, out=out, **a.args())
    assert got[0] is out and same(out.clone(), want[0]) and same(got[1], want[1])
    assert untouched(buf, offset, out.numel())


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("which", ["dq", "dk", "dv"])
def test_gradients(which, offset):
    """Through the C ABI, one of the three results at an odd place at a time."""
    t = torch()
    announce(f"linattn {which} {offset} elements on")
    b, L, hk, h, dk, dv = 1, 70, 1, 2, 64, 64
    a = Attention(b, L, hk, h, dk, dv, "bf16", "token", None, True, seed=32)
    q, k, v = (x.contiguous() for x in (a.q, a.k, a.v))
    want = ssm.linattn_backward(q, k, v, a.dout, dfinal=a.ds, **a.args())
    bufs = {n: odd(want[n].shape, offset if n == which else 0) for n in ("dq", "dk", "dv")}
    dg, di = t.empty_like(a.g), t.empty_like(a.s0)
    need = ssm.ssm_linattn_bwd_workspace_bytes(b, L, h, dk, dv, ssm.SSM_IO_BF16)
    ws = t.empty(need, dtype=t.uint8, device="cuda")
    p = lambda x: ctypes.c_void_p(x.data_ptr())
    status = ssm.ssm_linattn_bwd(
        p(q), None, p(k), None, p(v), None, p(a.dout), None, p(a.g), None, p(a.s0), None, p(a.ds), dk ** -0.5,
        ssm.SSM_IO_BF16, *(p(bufs[n][0]) for n in ("dq", "dk", "dv")), p(dg), p(di), p(ws), need, b, L, hk, h, dk, dv,
        t.cuda.current_stream().cuda_stream)
    assert status == ssm.SSM_OK
    t.cuda.synchronize()
    for n, (view, buf) in bufs.items():
        assert same(view.clone(), want[n]), n
        assert untouched(buf, offset if n == which else 0, view.numel()), n
    assert same(dg, want["dg"]) and same(di, want["dinitial"])
