"""Steps of the queries' and keys' norm that are padding (a position below 0) on the device: zeros and no
gradient, with a rotation and without one."""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import Rand, same
from gpu_util import announce, torch
from selective_state_space_fwd_amd import block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("L", [9, 3000])  # (3000 steps of 12 heads: a large call)
def test_padding(L, rot, io, native, monkeypatch):
    t = torch()
    announce(f"qk_norm padding L{L} rot {rot} {io} {native}")
    block._load()
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    r = Rand(90)
    b, hq, hk, d = 4, 8, 4, 64
    q, k, gq, gk = (r((b, L, n, d), io)[0] for n in (hq, hk, hq, hk))
    w = r((d,))[0]
    angle = t.rand(L + 8, 16, device="cuda")
    opt = dict(cos=angle.cos(), sin=angle.sin()) if rot else {}
    at = (t.arange(L)[None] + t.tensor([[0], [5], [2], [0]])).to(t.int32).cuda()
    pad = t.zeros(b, L, dtype=t.bool, device="cuda")
    pad[0, 7:], pad[2, 0], pad[3] = True, True, True
    # the padding's values 0: no part of the weights' gradients
    clean = [t.where(pad[..., None, None], t.zeros_like(x), x) for x in (q, k, gq, gk)]
    want = ssm.qk_norm(clean[0], clean[1], w, w, positions=at, **opt)
    grads = ssm.qk_norm_backward(*clean, w, w, positions=at, **opt)
    for x, bad in ((q, "nan"), (k, "inf"), (gq, "nan"), (gk, "nan")):
        x[pad] = float(bad)
    at[pad] = t.randint(-2 ** 31, 0, (int(pad.sum()),), device="cuda").to(t.int32)
    at[0, 7:], at[2, 0] = -1, -1
    got = ssm.qk_norm(q, k, w, w, positions=at, **opt)
    d = ssm.qk_norm_backward(q, k, gq, gk, w, w, positions=at, **opt)
    assert all((x[pad] == 0).all() for x in (*got, d["dq"], d["dk"]))
    live = ~pad
    assert all(same(x[live], y[live]) for x, y in zip(got, want))
    assert all(same(d[n][live], grads[n][live]) for n in ("dq", "dk"))
    assert all(same(d[n], grads[n]) for n in ("dq_weight", "dk_weight"))
