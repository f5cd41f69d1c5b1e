"""Host-only checks of linear attention and of the queries' and keys' norm (include/ssm_linattn.h,
ssm_qk.h): every invalid call is refused with its documented status before any HIP call, empty
problems that launch nothing pass, the launch rules hold over all sizes, and the binding refuses
what it cannot marshal. No call here reaches a kernel launch."""
import ctypes
import os
import re
import subprocess

import pytest

import selective_state_space_fwd_amd as ssm
from selective_state_space_fwd_amd import block
from selective_state_space_fwd_amd.build import CSRC, INCLUDE

P = [0x10000000 * (i + 1) for i in range(24)]
BF, F32 = ssm.SSM_IO_BF16, ssm.SSM_IO_F32
INVALID, UNSUPPORTED, MISALIGNED = (ssm.SSM_ERR_INVALID_ARG, ssm.SSM_ERR_UNSUPPORTED, ssm.SSM_ERR_MISALIGNED)
BIG = 1 << 61


def st(*v):
    return (ctypes.c_int64 * len(v))(*v)


def refused(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_flag_constants_match_the_headers():
    for header, name in (("ssm_linattn.h", "SSM_LINATTN_HEAD_DG"), ("ssm_qk.h", "SSM_QK_INTERLEAVED")):
        m = re.search(rf"#define {name} \(1u << (\d+)\)", open(os.path.join(INCLUDE, header)).read())
        assert m and 1 << int(m.group(1)) == getattr(ssm, name)


SIZES = dict(batch=2, seqlen=8, qk_heads=2, heads=4, dk=16, dv=8, stream=None)
# what the sizes' common checks refuse
BAD_SIZES = [dict(batch=-1), dict(seqlen=-1), dict(qk_heads=-1), dict(heads=-1), dict(dk=-1), dict(dv=-1),
             dict(heads=5), dict(qk_heads=0), dict(heads=0)]
UNFIT = [dict(flags=2), dict(flags=3), dict(dk=0), dict(dv=0), dict(dk=257), dict(dv=257), dict(batch=1 << 16),
         dict(seqlen=1 << 31), dict(seqlen=(1 << 31) - 1, batch=60000, heads=1 << 20, qk_heads=1 << 20)]


def fwd(**kw):
    a = dict(q=P[0], qs=None, k=P[1], ks=None, v=P[2], vs=None, g=None, gs=None, s0=None, n=None, scale=0.5,
             flags=BF, out=P[3], fin=None, ws=P[4], wsb=1 << 30, **SIZES)
    a.update(kw)
    return ssm.ssm_linattn_fwd(*a.values())


def test_fwd_refusals():
    refused(fwd, INVALID, BAD_SIZES + [
        dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(flags=BF | 1 << 4),
        dict(flags=BF | ssm.SSM_LINATTN_HEAD_DG), dict(out=P[0]), dict(out=P[2] + 64), dict(fin=P[3]),
        dict(s0=P[5], fin=P[5]), dict(g=P[3]), dict(n=P[3]), dict(qs=st(-1, 32, 16)), dict(vs=st(256, -32, 8)),
        dict(gs=st(0, 0, -1), g=P[6]), dict(qs=st(P[3] - P[0], 32, 16)),
        dict(seqlen=500, ws=None), dict(seqlen=500, wsb=100), dict(seqlen=500, ws=P[3])])
    refused(fwd, UNSUPPORTED, UNFIT + [
        dict(qs=st(BIG, 32, 16), batch=9), dict(ks=st(1 << 40, 1 << 24, 16)), dict(gs=st(1 << 40, 1 << 23, 1), g=P[6]),
        dict(heads=1 << 17, qk_heads=1 << 17, dv=64), dict(heads=1 << 26, qk_heads=1 << 26, dv=1, dk=1, seqlen=1)])
    refused(fwd, MISALIGNED, [
        dict(q=P[0] + 1), dict(k=P[1] + 1), dict(v=P[2] + 1), dict(out=P[3] + 1), dict(g=P[6] + 2), dict(s0=P[6] + 1),
        dict(fin=P[6] + 2), dict(n=P[6] + 1), dict(flags=F32, q=P[0] + 2), dict(ws=P[4] + 16)])
    assert fwd(batch=0) == fwd(heads=0, qk_heads=0) == fwd(seqlen=0) == ssm.SSM_OK


def bwd(**kw):
    a = dict(q=P[0], qs=None, k=P[1], ks=None, v=P[2], vs=None, do=P[3], dos=None, g=P[4], gs=None, s0=None, n=None,
             ds=None, scale=0.5, flags=BF, dq=P[5], dk_=P[6], dv_=P[7], dg=P[8], di=None, ws=P[9], wsb=1 << 30, **SIZES)
    a.update(kw)
    return ssm.ssm_linattn_bwd(*a.values())


def test_bwd_refusals():
    need = ssm.ssm_linattn_bwd_workspace_bytes(2, 8, 4, 16, 8, BF)
    refused(bwd, INVALID, BAD_SIZES + [
        dict(q=None), dict(do=None), dict(dq=None), dict(dk_=None), dict(dv_=None), dict(g=None), dict(ws=None),
        dict(wsb=need - 1), dict(dq=P[0]), dict(dk_=P[5]), dict(dv_=P[3]), dict(dg=P[4]), dict(di=P[8], s0=P[10]),
        dict(ds=P[10], di=P[10]), dict(ws=P[7]), dict(dos=st(256, -32, 8)), dict(flags=BF | 1 << 12)])
    refused(bwd, UNSUPPORTED, UNFIT + [dict(dos=st(1 << 40, 1 << 24, 8))])
    refused(bwd, MISALIGNED, [dict(do=P[3] + 1), dict(dq=P[5] + 1), dict(dg=P[8] + 2), dict(di=P[10] + 1),
                              dict(ds=P[10] + 2), dict(ws=P[9] + 64)])
    assert bwd(heads=0, qk_heads=0) == bwd(batch=0) == ssm.SSM_OK


def step(**kw):
    a = dict(q=P[0], qs=None, k=P[1], ks=None, v=P[2], vs=None, g=P[3], gs=None, slots=P[4], scale=0.5, flags=BF,
             state=P[5], out=P[6], batch=2, nslots=4, qk_heads=2, heads=4, dk=16, dv=8, stream=None)
    a.update(kw)
    return ssm.ssm_linattn_step(*a.values())


def test_step_refusals():
    refused(step, INVALID, [
        dict(q=None), dict(v=None), dict(out=None), dict(state=None), dict(nslots=-1), dict(slots=None, nslots=1),
        dict(heads=5), dict(batch=-1), dict(out=P[5]), dict(state=P[0]), dict(out=P[4]), dict(qs=st(-32, 16)),
        dict(gs=st(-4, 1)), dict(flags=BF | 1 << 5)])
    refused(step, UNSUPPORTED, [dict(flags=3), dict(dk=257), dict(dv=0), dict(batch=1 << 16), dict(nslots=1 << 31),
                                dict(heads=1 << 25, qk_heads=1 << 25, dk=1, dv=1, nslots=4), dict(qs=st(BIG * 3, 16), batch=3)])
    refused(step, MISALIGNED, [dict(q=P[0] + 1), dict(state=P[5] + 2), dict(slots=P[4] + 1), dict(g=P[3] + 1)])
    assert step(batch=0) == step(heads=0, qk_heads=0) == ssm.SSM_OK


def qk(**kw):
    a = dict(q=P[0], qs=None, k=P[1], ks=None, qw=P[2], kw=None, cos=P[3], sin=P[4], pos=None, eps=1e-6, flags=BF,
             qo=P[5], ko=P[6], batch=2, seqlen=8, hq=4, hk=2, dim=16, rot=8, rows=8, stream=None)
    a.update(kw)
    return ssm.ssm_qk_norm_fwd(*a.values())


def qk_bwd(**kw):
    a = dict(q=P[0], qs=None, k=P[1], ks=None, gq=P[7], gqs=None, gk=P[8], gks=None, qw=P[2], kw=None, cos=P[3],
             sin=P[4], pos=None, eps=1e-6, flags=BF, dq=P[5], dk=P[6], dqw=P[9], dkw=P[10], ws=P[11], wsb=1 << 20,
             batch=2, seqlen=8, hq=4, hk=2, dim=16, rot=8, rows=8, stream=None)
    a.update(kw)
    return ssm.ssm_qk_norm_bwd(*a.values())


def test_qk_refusals():
    common = [dict(q=None), dict(k=None), dict(cos=None), dict(sin=None), dict(batch=-1), dict(hq=-1), dict(rot=-2),
              dict(rows=-1), dict(flags=BF | 1 << 13), dict(qs=st(-1, 64, 16))]
    unfit = [dict(dim=0), dict(dim=257), dict(rot=18), dict(rot=7), dict(flags=2), dict(seqlen=1 << 31),
             dict(batch=1 << 20, seqlen=1 << 20, hq=1 << 20, hk=0)]
    refused(qk, INVALID, common + [dict(qo=None), dict(ko=None), dict(qo=P[0]), dict(ko=P[5]), dict(qo=P[3]),
                                   dict(pos=P[5])])
    refused(qk, UNSUPPORTED, unfit)
    refused(qk, MISALIGNED, [dict(q=P[0] + 1), dict(qw=P[2] + 2), dict(cos=P[3] + 1), dict(pos=P[12] + 2), dict(qo=P[5] + 1)])
    assert qk(batch=0) == qk(seqlen=0) == qk(hq=0, hk=0) == ssm.SSM_OK
    need = ssm.ssm_qk_norm_bwd_workspace_bytes(2, 8, 4, 2, 16, 8, BF)
    refused(qk_bwd, INVALID, common + [dict(gq=None), dict(dq=None), dict(dk=None), dict(ws=None), dict(wsb=need - 1),
                                       dict(dq=P[7]), dict(dqw=P[2]), dict(dkw=P[9]), dict(ws=P[5])])
    refused(qk_bwd, UNSUPPORTED, unfit)
    refused(qk_bwd, MISALIGNED, [dict(gk=P[8] + 1), dict(dqw=P[9] + 2), dict(ws=P[11] + 4)])


def test_workspaces():
    f, b = ssm.ssm_linattn_fwd_workspace_bytes, ssm.ssm_linattn_bwd_workspace_bytes
    assert f(16, 2048, 32, 128, 64, BF) == 0          # 512 workgroups of whole rows
    assert f(4, 2048, 32, 128, 64, BF) == 4 * 32 * 4 * (128 * 64 + 1) * 4  # four segments
    # b3, 4 heads of 64 x 100 (padded to 128), 17 chunks of 32 steps, joined
    assert b(3, 517, 4, 64, 100, F32) == 3 * 4 * 17 * (2 * 64 * 128 + 4) * 4
    for w in (f, b):
        assert w(-1, 1, 1, 1, 1, BF) == w(1, 1, 1, 257, 1, BF) == w(1, 1, 1, 1, 1, 3) == -1
        assert w(1 << 15, 1 << 30, 1 << 20, 256, 256, BF) == -1
        assert w(0, 5, 4, 16, 16, BF) == 0


def test_launch_rules(tmp_path):
    """The segments, walks and grids over a range of sizes: every chunk once, no empty segment, the
    workspace's parts inside it. (linattn_launch.h, compiled by the host's compiler.)"""
    source = tmp_path / "rules.cpp"
    source.write_text(r"""
#include <stdio.h>
#include "linattn_launch.h"
#include "qk_launch.h"
using namespace ssm;
int main() {
  int bad = 0;
  for (int64_t b : {1, 2, 3, 16, 400, 65535}) for (int64_t h : {1, 2, 5, 32, 96}) for (int64_t k : {1, 64, 100, 129, 256})
  for (int64_t v : {1, 64, 65, 128, 200}) for (int64_t L : {0, 1, 31, 32, 33, 64, 65, 1000, 4097, 65536, 1 << 22})
  for (Io io : {Io::F32, Io::BF16}) {
    const int64_t c = linattn_chunk(io), cb = linattn_bwd_chunk(io, k, v);
    const LinattnSegments s = linattn_segments(b, h, k, v, L, io);
    bad += s.chunks != (L + c - 1) / c || s.per < 1 || s.count < 1;
    bad += L > 0 && (s.per * s.count < s.chunks || s.per * (s.count - 1) >= s.chunks);
    const LinattnBwdStates w = linattn_bwd_states(b, h, k, v, L, io);
    bad += w.chunks != (L + cb - 1) / cb || w.floats % 4 || w.floats < k * v || w.total < w.chunk_rows * (2 * w.floats + 2);
    if (w.walked) {
      bad += w.segments.per * w.segments.count < w.chunks || w.segments.per * (w.segments.count - 1) >= w.chunks;
      bad += w.segments.count > 1 && w.segment_rows != b * h * w.segments.count;
      bad += w.total < (w.chunk_rows + w.segment_rows) * (2 * w.floats + 2);
    }
    const LinattnStepForm f = linattn_step_form(h, k, v);
    bad += f.tiles * kLinattnStepWaves * f.rows * (64 >> step_lanes_log2(k)) < v || f.rows * (64 >> step_lanes_log2(k)) > 64;
  }
  for (int64_t d = 1; d <= 256; ++d) for (int64_t r = 0; r <= d; r += 2) {
    const int lg = qk_lanes_log2(d, r);
    bad += lg > 6 || (1 << lg) < qk_units(d, r);
  }
  printf("%d wrong\n", bad);
  return bad != 0;
}
""")
    exe = str(tmp_path / "rules")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", INCLUDE, "-o", exe, str(source)], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("native", [True, False])
def test_binding_refuses_host_tensors(native, monkeypatch):
    t = pytest.importorskip("torch")
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    x, s = t.zeros(1, 4, 2, 8), t.zeros(1, 2, 8, 8)
    for call in (lambda: ssm.linattn(x, x, x), lambda: ssm.linattn_backward(x, x, x, x),
                 lambda: ssm.linattn_step(x[:, 0], x[:, 0], x[:, 0], s), lambda: ssm.qk_norm(x, x),
                 lambda: ssm.qk_norm_backward(x, x, x, x), lambda: ssm.linear_attention(x, x, x),
                 lambda: ssm.rotary_qk_norm(x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="must be"):
        ssm.linattn(x[0], x[0], x[0])
    with pytest.raises(ValueError, match="multiple|device"):
        ssm.linattn(x, x, t.zeros(1, 4, 3, 8))
