"""Head sizes that linear attention does not take are refused alike by both ways of marshalling a call."""
import pytest

import selective_state_space_fwd_amd as ssm
from gpu_util import announce, torch
from selective_state_space_fwd_amd import block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("dk,dv", [(0, 8), (8, 0), (257, 8), (8, 257)])
def test_refused(dk, dv, native, monkeypatch):
    t = torch()
    announce(f"linattn {dk}x{dv} refused, native {native}")
    block._load()
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    q, v = t.zeros(1, 4, 2, dk, device="cuda"), t.zeros(1, 4, 2, dv, device="cuda")
    state = t.zeros(1, 2, dv, dk, device="cuda")
    for call in (lambda: ssm.linattn(q, q, v), lambda: ssm.linattn_backward(q, q, v, v),
                 lambda: ssm.linattn_step(q[:, 0], q[:, 0], v[:, 0], state), lambda: ssm.linear_attention(q, q, v)):
        with pytest.raises(ssm.SsmScanError):
            call()
