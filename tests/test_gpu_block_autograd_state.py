"""What the operators around the scan write in place (caches, results given by the caller) counts as
written for autograd: a backward pass that needs the value from before refuses instead of using
the new one. Both ways of marshalling a call."""
import pytest

import selective_state_space_fwd_amd as ssm
from gpu_util import announce, torch
from selective_state_space_fwd_amd import block

pytestmark = pytest.mark.gpu


def calls():
    """(name, the tensors it writes, the call)."""
    t = torch()
    g = t.Generator().manual_seed(5)
    mk = lambda *s: t.randn(s, generator=g).cuda()
    x, w, xs = mk(2, 8), mk(8, 4), mk(2, 8, 16)
    A, B, cs, st = -mk(8, 4).abs(), mk(2, 4), mk(2, 8, 3), mk(2, 8, 4)
    st2, o1, o2, o3, o4, fin = mk(2, 8, 4), mk(2, 8), mk(2, 8), mk(2, 8, 16), mk(2, 16, 8), mk(2, 8, 3)
    return [("conv_step", [cs, o1], lambda: ssm.conv_step(x, cs, w, out=o1)),
            ("scan_step", [st, o2], lambda: ssm.scan_step(x, x, A, B, B, st, out=o2)),
            ("ssd_step", [st2], lambda: ssm.ssd_step(x, x[:, :2].contiguous(), A[:2, 0].contiguous(), B, B, st2)),
            ("conv", [o3, fin], lambda: ssm.conv(xs, w, out=o3, final_state=fin)),
            ("norm", [o4], lambda: ssm.norm(xs, w[:, 0].contiguous(), token_major=True, out=o4))]


@pytest.mark.parametrize("native", [True, False])
def test_writes_are_seen_by_autograd(native, monkeypatch):
    announce(f"writes seen by autograd, module {native}")
    t = torch()
    block._load()
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    for name, written, call in calls():
        for v in written:
            scale = t.ones_like(v, requires_grad=True)
            loss = (v * scale).sum()
            call()
            with pytest.raises(RuntimeError, match="inplace operation"):
                loss.backward()
    with t.inference_mode():  # tensors that have no version
        for name, written, call in calls():
            call()
        frozen = calls()
    for name, written, call in frozen:
        call()
