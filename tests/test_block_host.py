"""Host-only checks of the operators around the scan (include/ssm_conv.h, ssm_step.h,
ssm_norm.h): every invalid call is refused with its documented status before any HIP call,
empty problems that launch nothing pass, and the binding refuses what it cannot marshal.

No call here reaches a kernel launch, so the addresses are never dereferenced.
"""
import ctypes
import os
import re

import pytest

import selective_state_space_fwd_amd as ssm
from selective_state_space_fwd_amd.build import INCLUDE

# fake, well-separated, 256-byte aligned addresses
P = [0x10000000 * (i + 1) for i in range(24)]
BF, F32 = ssm.SSM_IO_BF16, ssm.SSM_IO_F32
BIG = 1 << 62


def st(*v):
    return (ctypes.c_int64 * 3)(*v)


def refused(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_flag_constants_match_the_headers():
    for header, name in (("ssm_conv.h", "SSM_CONV_SILU"), ("ssm_norm.h", "SSM_NORM_BEFORE_GATE")):
        m = re.search(rf"#define {name} \(1u << (\d+)\)", open(os.path.join(INCLUDE, header)).read())
        assert m and 1 << int(m.group(1)) == getattr(ssm, name)


# ---------------------------------------------------------------- convolution

def conv(**kw):
    a = dict(x=P[0], xs=None, w=P[1], bias=None, init=None, lengths=None, flags=BF, out=P[2],
             fin=None, batch=2, dim=4, width=4, seqlen=8, stream=None)
    a.update(kw)
    return ssm.ssm_conv_fwd(*a.values())


def test_conv_refusals():
    refused(conv, ssm.SSM_ERR_INVALID_ARG, [
        dict(x=None), dict(w=None), dict(out=None), dict(batch=-1), dict(dim=-1),
        dict(seqlen=-1), dict(width=-1), dict(flags=BF | 1 << 4), dict(flags=BF | 1 << 12),
        dict(out=P[0]), dict(out=P[0] + 64), dict(out=P[1]), dict(fin=P[2]), dict(fin=P[0]),
        dict(init=P[3], fin=P[3]), dict(lengths=P[2]), dict(xs=st(-32, 8, 1)),
        dict(xs=st(1 << 30, 1, -4)), dict(xs=st(P[2] - P[0], 8, 1))])  # x reaches over out
    refused(conv, ssm.SSM_ERR_UNSUPPORTED, [
        dict(flags=2), dict(flags=3), dict(width=1), dict(width=5), dict(width=0),
        dict(xs=st(64, 16, 2)), dict(batch=1 << 20, dim=1 << 12), dict(seqlen=1 << 31),
        dict(batch=1 << 16, dim=1 << 15, seqlen=1 << 20), dict(xs=st(BIG, 8, 1), batch=5),
        dict(dim=1 << 30)])
    refused(conv, ssm.SSM_ERR_MISALIGNED, [
        dict(x=P[0] + 1), dict(out=P[2] + 1), dict(w=P[1] + 2), dict(bias=P[3] + 1),
        dict(init=P[3] + 1), dict(fin=P[3] + 1), dict(lengths=P[3] + 2),
        dict(flags=F32, x=P[0] + 2)])
    assert conv(batch=0) == conv(dim=0) == conv(seqlen=0) == ssm.SSM_OK


def conv_bwd(**kw):
    a = dict(x=P[0], xs=None, w=P[1], bias=None, init=None, lengths=None, flags=BF, dout=P[2],
             dfin=None, dx=P[3], dxs=None, dw=P[4], db=None, di=None, ws=P[5], wsb=1 << 20,
             batch=2, dim=4, width=4, seqlen=8, stream=None)
    a.update(kw)
    return ssm.ssm_conv_bwd(*a.values())


def test_conv_bwd_refusals():
    need = ssm.ssm_conv_bwd_workspace_bytes(2, 4, 4, 8, BF)
    refused(conv_bwd, ssm.SSM_ERR_INVALID_ARG, [
        dict(x=None), dict(dout=None), dict(dx=None), dict(dw=None), dict(ws=None),
        dict(wsb=need - 1), dict(ws=P[3]), dict(dx=P[2]), dict(dx=P[0]), dict(db=P[4]),
        dict(di=P[3]), dict(dw=P[1]), dict(dxs=st(8, 8, 1)), dict(dxs=st(0, 8, 1)),
        dict(dxs=st(32, 4, 1)), dict(flags=BF | 1 << 10)])
    refused(conv_bwd, ssm.SSM_ERR_UNSUPPORTED, [
        dict(dxs=st(32, 1, 4)), dict(xs=st(32, 1, 4)), dict(width=6), dict(flags=2)])
    refused(conv_bwd, ssm.SSM_ERR_MISALIGNED, [
        dict(ws=P[5] + 16), dict(dx=P[3] + 1), dict(dw=P[4] + 2), dict(dout=P[2] + 1)])
    assert conv_bwd(dim=0) == ssm.SSM_OK


def test_conv_workspace():
    ws = ssm.ssm_conv_bwd_workspace_bytes
    # a row of 2048 bf16 steps: runs of 128 steps with channels contiguous (of 2048 else)
    assert ws(4, 2304, 4, 2048, BF) == 4 * 16 * 2304 * 5 * 4
    assert ws(3, 10, 2, 1, F32) == 3 * 10 * 3 * 4
    assert ws(3, 10, 2, 0, F32) == 3 * 10 * 3 * 4 and ws(0, 10, 2, 5, F32) == 0
    for bad in ((-1, 1, 4, 1, BF), (1, -1, 4, 1, BF), (1, 1, 4, -1, BF), (1, 1, 1, 1, BF),
                (1, 1, 5, 1, BF), (1, 1, 4, 1, 2), (1 << 40, 1 << 40, 4, 1, BF),
                (1 << 30, BIG, 4, 1 << 30, BF)):
        assert ws(*bad) == -1, bad


def conv_step(**kw):
    a = dict(x=P[0], xs=4, state=P[1], w=P[2], bias=None, slots=None, flags=BF, out=P[3],
             batch=2, nslots=2, dim=4, width=4, stream=None)
    a.update(kw)
    return ssm.ssm_conv_step(*a.values())


def test_conv_step_refusals():
    refused(conv_step, ssm.SSM_ERR_INVALID_ARG, [
        dict(x=None), dict(state=None), dict(w=None), dict(out=None), dict(nslots=1),
        dict(nslots=-1), dict(batch=-1), dict(xs=-4), dict(out=P[0]), dict(out=P[1]),
        dict(state=P[0]), dict(state=P[2]), dict(slots=P[1]), dict(flags=BF | 1 << 5)])
    refused(conv_step, ssm.SSM_ERR_UNSUPPORTED, [
        dict(width=1), dict(width=5), dict(batch=65536, nslots=65536), dict(nslots=1 << 31, slots=P[5]),
        dict(flags=3), dict(xs=BIG, batch=2), dict(dim=1 << 31)])
    refused(conv_step, ssm.SSM_ERR_MISALIGNED, [
        dict(x=P[0] + 1), dict(state=P[1] + 1), dict(slots=P[5] + 2), dict(w=P[2] + 2)])
    assert conv_step(batch=0) == conv_step(dim=0) == ssm.SSM_OK


# ---------------------------------------------------------------- state steps

def scan_step(**kw):
    a = dict(u=P[0], us=4, dt=P[1], dts=4, A=P[2], B=P[3], bs=16, C=P[4], cs=16, D=None, z=None,
             zs=0, bias=None, slots=None, flags=BF, state=P[5], out=P[6], batch=2, nslots=2,
             dim=4, dstate=16, stream=None)
    a.update(kw)
    return ssm.ssm_scan_step(*a.values())


def ssd_step(**kw):
    a = dict(x=P[0], xs=8, dt=P[1], dts=2, A=P[2], B=P[3], bs=16, C=P[4], cs=16, D=None, z=None,
             zs=0, bias=None, slots=None, flags=BF, state=P[5], out=P[6], batch=2, nslots=2,
             heads=2, headdim=4, dstate=16, stream=None)
    a.update(kw)
    return ssm.ssm_ssd_step(*a.values())


@pytest.mark.parametrize("call", [scan_step, ssd_step])
def test_step_refusals(call):
    refused(call, ssm.SSM_ERR_INVALID_ARG, [
        dict(dt=None), dict(A=None), dict(B=None), dict(C=None), dict(state=None),
        dict(out=None), dict(nslots=1), dict(nslots=-1), dict(batch=-1), dict(dstate=-1),
        dict(bs=-1), dict(z=P[7], zs=-4), dict(out=P[0]), dict(out=P[5]), dict(state=P[3]),
        dict(state=P[2]), dict(slots=P[5]), dict(flags=BF | 1 << 5), dict(D=P[6])])
    refused(call, ssm.SSM_ERR_UNSUPPORTED, [
        dict(dstate=0), dict(dstate=257), dict(flags=2), dict(batch=65536, nslots=65536),
        dict(nslots=1 << 31, slots=P[8]), dict(cs=BIG), dict(dts=BIG)])
    refused(call, ssm.SSM_ERR_MISALIGNED, [
        dict(dt=P[1] + 1), dict(A=P[2] + 2), dict(state=P[5] + 2), dict(D=P[7] + 2),
        dict(z=P[7] + 1, zs=8), dict(bias=P[7] + 1), dict(slots=P[7] + 2), dict(out=P[6] + 1)])
    assert call(batch=0) == ssm.SSM_OK


def test_step_sizes():
    assert ssd_step(headdim=0) == ssm.SSM_ERR_UNSUPPORTED
    assert ssd_step(heads=1 << 20, headdim=1 << 20) == ssm.SSM_ERR_UNSUPPORTED
    assert ssd_step(heads=-1) == ssd_step(headdim=-1) == ssm.SSM_ERR_INVALID_ARG
    assert ssd_step(heads=0, A=None) == scan_step(dim=0) == ssm.SSM_OK
    assert scan_step(dim=1 << 31) == ssm.SSM_ERR_UNSUPPORTED


# ---------------------------------------------------------------- norm

def norm(**kw):
    a = dict(y=P[0], ys=None, z=None, zs=None, w=P[1], eps=1e-5, flags=BF, out=P[2], os=None,
             rstd=None, ws=P[9], wsb=1 << 20, batch=2, dim=4, groups=1, seqlen=8, stream=None)
    a.update(kw)
    return ssm.ssm_norm_fwd(*a.values())


def test_norm_refusals():
    refused(norm, ssm.SSM_ERR_INVALID_ARG, [
        dict(y=None), dict(w=None), dict(out=None), dict(batch=-1), dict(dim=-1),
        dict(seqlen=-1), dict(groups=0), dict(groups=3), dict(eps=-1.0), dict(eps=float("nan")),
        dict(flags=BF | 1 << 11), dict(out=P[0]), dict(z=P[2]), dict(rstd=P[2]), dict(rstd=P[1]),
        dict(os=st(8, 8, 1)), dict(os=st(32, 1, 3)), dict(ys=st(-1, 8, 1)), dict(ws=None),
        dict(wsb=0), dict(ws=P[0]),
        dict(wsb=ssm.ssm_norm_fwd_workspace_bytes(2, 4, 1, 8, BF) - 1)])
    refused(norm, ssm.SSM_ERR_UNSUPPORTED, [
        dict(flags=2), dict(ys=st(64, 16, 2)), dict(z=P[3], zs=st(64, 16, 2)),
        dict(os=st(64, 16, 2)), dict(batch=1 << 20, seqlen=1 << 20), dict(seqlen=1 << 31),
        dict(batch=1 << 31, seqlen=1)])
    refused(norm, ssm.SSM_ERR_MISALIGNED, [
        dict(y=P[0] + 1), dict(z=P[3] + 1), dict(out=P[2] + 1), dict(w=P[1] + 2),
        dict(rstd=P[3] + 2), dict(ws=P[9] + 64)])
    ws = ssm.ssm_norm_fwd_workspace_bytes
    assert ws(2, 4, 1, 8, BF) == 2 * 8 * 4 and ws(3, 1024, 2, 5, F32) == 3 * 2 * 4 * 5 * 4
    assert ws(0, 4, 1, 8, BF) == 0 and ws(1, 4, 3, 8, BF) == ws(1, -4, 1, 8, BF) == -1
    assert norm(batch=0) == norm(dim=0) == norm(seqlen=0) == ssm.SSM_OK


def norm_bwd(**kw):
    a = dict(y=P[0], ys=None, z=P[1], zs=None, w=P[2], rstd=P[3], dout=P[4], gs=None, flags=BF,
             dy=P[5], dys=None, dz=P[6], dzs=None, dw=P[7], ws=P[8], wsb=1 << 20, batch=2, dim=4,
             groups=1, seqlen=8, stream=None)
    a.update(kw)
    return ssm.ssm_norm_bwd(*a.values())


def test_norm_bwd_refusals():
    need = ssm.ssm_norm_bwd_workspace_bytes(2, 4, 1, 8, BF)
    assert need > 0
    refused(norm_bwd, ssm.SSM_ERR_INVALID_ARG, [
        dict(y=None), dict(rstd=None), dict(dout=None), dict(dy=None), dict(dz=None),
        dict(dw=None), dict(ws=None), dict(wsb=need - 1), dict(dy=P[0]), dict(dz=P[5]),
        dict(dw=P[2]), dict(ws=P[3]), dict(dys=st(0, 8, 1)), dict(dzs=st(8, 1, 4))])
    refused(norm_bwd, ssm.SSM_ERR_UNSUPPORTED, [dict(flags=3), dict(gs=st(64, 16, 2))])
    refused(norm_bwd, ssm.SSM_ERR_MISALIGNED, [
        dict(ws=P[8] + 64), dict(dy=P[5] + 1), dict(dz=P[6] + 1), dict(dw=P[7] + 2)])
    assert norm_bwd(dim=0) == ssm.SSM_OK
    ws = ssm.ssm_norm_bwd_workspace_bytes
    assert ws(0, 4, 1, 8, BF) == ws(2, 4, 1, 0, BF) == 0
    for bad in ((-1, 4, 1, 8, BF), (1, 4, 3, 8, BF), (1, 4, 0, 8, BF), (1, 4, 1, 8, 2),
                (1 << 31, 4, 1, 8, BF)):
        assert ws(*bad) == -1, bad


# ---------------------------------------------------------------- binding

def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    t = pytest.importorskip("torch")
    x, w = t.zeros(1, 2, 8), t.zeros(2, 4)
    for call in (lambda: ssm.conv(x, w), lambda: ssm.conv_backward(x, w, x),
                 lambda: ssm.causal_conv(x, w), lambda: ssm.norm(x, w[:, 0]),
                 lambda: ssm.gated_norm(x, w[:, 0]),
                 lambda: ssm.norm_backward(x, w[:, 0], x, x),
                 lambda: ssm.conv_step(x[0], x, w),
                 lambda: ssm.scan_step(x[0], x[0], w, w, w, x),
                 lambda: ssm.ssd_step(x[0], x[0], w[:, 0], w, w, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        ssm.scan_step(x[0], x[0], w[:, 0], w, w, x)   # A of Mamba-2
    with pytest.raises(ValueError):
        ssm.ssd_step(x[0], x[0], w, w, w, x)          # A of Mamba-1
    with pytest.raises(ValueError):
        ssm.ssd_step(x[0], x[0], t.zeros(3), w, w, x)  # 8 channels of 3 heads
