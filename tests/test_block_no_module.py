"""Without the binding's extension module (_binding.so): the library's build, which needs hipcc alone,
does not depend on it, and the operators around the scan marshal every call in Python."""
import sys

import pytest

import selective_state_space_fwd_amd as ssm
from selective_state_space_fwd_amd import block
from selective_state_space_fwd_amd import build as hip_build


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """build() with its compiles recorded instead, and a module's file left by an earlier build."""
    made = []
    left = tmp_path / "_binding.so"
    left.write_bytes(b"old")
    monkeypatch.setattr(hip_build, "BINDING_PATH", str(left))
    monkeypatch.setattr(hip_build, "_link", lambda sources, target, *a: made.append(target))
    monkeypatch.setattr(hip_build, "_compile", lambda cmd, sources, target, v: made.append(target))
    return made, left


LIBRARIES = [hip_build.PROBE_LIB_PATH, hip_build.SHAPE2_LIB_PATH, hip_build.LIB_PATH]


def test_build_makes_the_module_last(steps):
    made, left = steps
    assert hip_build.build() == hip_build.LIB_PATH
    assert made == LIBRARIES + [str(left)]


def test_build_without_a_compiler(steps, monkeypatch):
    made, left = steps
    monkeypatch.setenv("CXX", "no-such-compiler")
    with pytest.warns(UserWarning, match="no-such-compiler"):
        assert hip_build.build() == hip_build.LIB_PATH
    assert made == LIBRARIES and not left.exists()


def test_build_without_torch(steps, monkeypatch):
    made, left = steps
    monkeypatch.setitem(sys.modules, "torch.utils.cpp_extension", None)
    with pytest.warns(UserWarning, match="no torch"):
        assert hip_build.build() == hip_build.LIB_PATH
    assert made == LIBRARIES and not left.exists()


def test_build_without_headers(steps, monkeypatch):
    made, _ = steps
    import torch.utils.cpp_extension as ext
    monkeypatch.setattr(ext, "include_paths", lambda *a, **k: ["/no/such/place"])
    with pytest.warns(UserWarning, match="headers"):
        hip_build.build()
    assert made == LIBRARIES


def test_a_module_that_does_not_compile_is_an_error(steps, monkeypatch):
    made, _ = steps

    def fails(*a):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(hip_build, "_compile", fails)
    with pytest.raises(RuntimeError, match="g[+][+] failed"):
        hip_build.build()
    assert made == LIBRARIES


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    monkeypatch.setattr(block, "BINDING_PATH", str(tmp_path / "none.so"))
    monkeypatch.setattr(block, "_bound", None)
    monkeypatch.setattr(block, "_binding", None)


def test_calls_without_the_module(no_module):
    t = pytest.importorskip("torch")
    with pytest.warns(UserWarning, match="missing"):
        assert ssm.ssm_conv_bwd_workspace_bytes(0, 10, 2, 5, ssm.SSM_IO_F32) == 0
    x, w = t.zeros(1, 2, 8), t.zeros(2, 4)
    for call in (lambda: ssm.conv(x, w), lambda: ssm.conv_backward(x, w, x), lambda: ssm.norm(x, w[:, 0]),
                 lambda: ssm.norm_backward(x, w[:, 0], x, x), lambda: ssm.conv_step(x[0], x, w),
                 lambda: ssm.scan_step(x[0], x[0], w, w, w, x), lambda: ssm.ssd_step(x[0], x[0], w[:, 0], w, w, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


@pytest.mark.gpu
def test_results_without_the_module(monkeypatch, tmp_path):
    import torch as t
    print("\n[gpu-case] no module", flush=True)
    g = t.Generator().manual_seed(3)
    mk = lambda *s: t.randn(s, generator=g).cuda()
    x, w, cache = mk(2, 24, 40).bfloat16(), mk(24, 4), mk(2, 24, 3).bfloat16()

    def calls():
        c = cache.clone()
        d = ssm.conv_backward(x, w, x)
        return [*ssm.conv(x, w, silu=True), ssm.conv_step(x[:, :, 0].contiguous(), c, w), c, d["dx"], d["dweight"],
                ssm.norm(x, w[:, 0].contiguous(), z=x, token_major=True)]
    with_it = calls()
    monkeypatch.setattr(block, "BINDING_PATH", str(tmp_path / "none.so"))
    monkeypatch.setattr(block, "_bound", None)
    monkeypatch.setattr(block, "_binding", None)
    with pytest.warns(UserWarning, match="missing"):
        without = calls()
    assert block._binding is block._NoModule
    assert all(t.equal(a, b) for a, b in zip(with_it, without))


def test_built_files_are_readable_by_others(tmp_path, monkeypatch):
    """What the compilers write goes by the umask, also where they write into the file they are given
    (made for its owner alone)."""
    import os
    import shutil

    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("gcc not available")
    source, target = tmp_path / "one.c", tmp_path / "one.so"
    source.write_text("int one(void) { return 1; }\n")
    monkeypatch.setattr(hip_build, "PKG", str(tmp_path))
    before = os.umask(0o022)
    try:
        hip_build._compile([cc, "-fPIC"], [str(source)], str(target), False)
    finally:
        os.umask(before)
    assert target.stat().st_mode & 0o777 == 0o755
    assert sorted(p.name for p in tmp_path.iterdir()) == ["one.c", "one.so"]
