"""The calls of linear attention and of the queries' and keys' norm go through the extension module where their
arguments are what the C ABI takes as they stand."""
import pytest

import selective_state_space_fwd_amd as ssm
from gpu_util import announce, torch
from selective_state_space_fwd_amd import block
from test_gpu_linattn_together import every_call

pytestmark = pytest.mark.gpu
FUNCTIONS = ("linattn", "linattn_backward", "linattn_step", "qk_norm", "qk_norm_backward")


class Recorder:
    """The module, with (name, whether it made the call) of each call."""

    def __init__(self, module):
        self.module, self.made = module, []

    def __getattr__(self, name):
        fn = getattr(self.module, name)
        if name not in FUNCTIONS:
            return fn

        def call(*args):
            r = fn(*args)
            self.made.append((name, r is not None))
            return r

        return call


@pytest.fixture
def recorder(monkeypatch):
    module = block._load()
    assert module is not block._NoModule, "the extension module is not built"
    r = Recorder(module)
    monkeypatch.setattr(block, "_binding", r)
    return r


def test_the_module_makes_the_calls(recorder):
    announce("linattn calls through the extension module")
    names = set()
    for i, (_, call) in enumerate(every_call()):
        del recorder.made[:]
        call()
        assert len(recorder.made) == 1 and recorder.made[0][1], (i, recorder.made)
        names.add(recorder.made[0][0])
    assert names == set(FUNCTIONS)


def test_the_module_leaves_the_others(recorder):
    """An argument that has to be copied: made by the checks in Python, once."""
    t = torch()
    announce("linattn calls that the extension module leaves")
    q, v = t.randn(1, 8, 16, 2, device="cuda").transpose(2, 3), t.randn(1, 8, 2, 8, device="cuda")
    ssm.linattn(q, q, v)
    ssm.linattn_backward(q, q, v, v)
    ssm.qk_norm(q, q)
    ssm.linattn_step(q[:, 0], q[:, 0], v[:, 0], t.zeros(1, 2, 8, 16, device="cuda"))
    assert recorder.made == [("linattn", False), ("linattn_backward", False), ("qk_norm", False), ("linattn_step", False)]
