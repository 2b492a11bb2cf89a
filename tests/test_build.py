"""What a build needs: nvcc for the library, and torch and two sets of headers for the short way into some calls, without which
the library is built all the same.  The compilers here are stand-ins that write their outputs."""
import os
import types
import warnings

import pytest

import paged_kv_cache_201_gb300 as pa
from paged_kv_cache_201_gb300 import build as b


@pytest.fixture
def built(monkeypatch, tmp_path):
    """Builds into a folder of its own; the commands that ran."""
    for name in ("LIB_PATH", "BINDING_PATH", "BINDING_FOR"):
        if hasattr(b, name):
            monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(b.subprocess, "run", run)
    return ran


def _binding_ran(ran):
    return any(b.BINDING_SRC in c for c in ran)


def _without_torch(monkeypatch):
    find = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_without_torch(built, monkeypatch):
    _without_torch(monkeypatch)
    assert b.build(force=True) == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert not _binding_ran(built) and not os.path.exists(b.BINDING_PATH) and b.up_to_date()


def test_library_without_headers(built, monkeypatch, tmp_path):
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "nowhere")})
    assert b.build(force=True) == b.LIB_PATH and os.path.exists(b.LIB_PATH) and not _binding_ran(built)


def test_another_torch_builds_again(built, monkeypatch):
    b.build(force=True)
    assert _binding_ran(built) and b.up_to_date() and b.binding_fits()
    version = b.importlib.metadata.version
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "9.9" if name == "torch" else version(name))
    assert not b.binding_fits() and not b.up_to_date()
    built.clear()
    b.build()
    assert _binding_ran(built) and b.binding_fits() and b.up_to_date()


def test_an_old_binding_does_not_meet_a_new_library(built, monkeypatch):
    b.build(force=True)
    assert b.binding_fits()
    with monkeypatch.context() as m:  # its headers are gone
        m.setattr(b.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
        b.build(force=True)
        assert not b.binding_fits()
    b.build()
    assert b.binding_fits()
    run = b.subprocess.run  # or it does not compile
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no")
                        if b.BINDING_SRC in cmd else run(cmd, **kw))
    with pytest.raises(RuntimeError):
        b.build(force=True)
    assert not b.binding_fits()


def test_a_library_that_fails_says_so(built, monkeypatch):
    """Whatever becomes of the short way, a kernel that does not compile is an error."""
    _without_torch(monkeypatch)
    monkeypatch.setattr(b.subprocess, "run",
                        lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no"))
    with pytest.raises(RuntimeError):
        b.build(force=True)


def test_calls_without_the_short_way(monkeypatch, tmp_path):
    """They go the long way, with the same refusals, and say once that they do."""
    from tests.test_serving_step_abi import FakeCuda
    b.build()
    pa.load_library()
    monkeypatch.setattr(pa, "_binding", None)
    monkeypatch.setattr(b, "BINDING_FOR", str(tmp_path / "none"))
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(pa, "_stream", lambda s: None)
    u8 = torch.uint8
    with pytest.warns(RuntimeWarning, match="short way"):
        with pytest.raises(pa.PagedAttnError):  # reaches the library, which has no head_dim 96
            pa.paged_attn_gather_kv4(FakeCuda(9, 2, 9 * 16 * 96 // 8, dtype=u8), FakeCuda(5),
                                     FakeCuda(5, 2, 96, dtype=torch.bfloat16), FakeCuda(5, 2, 96, dtype=torch.bfloat16))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError):
            pa.paged_attn_gather_kv4(FakeCuda(9, 2, 1, dtype=u8), FakeCuda(5), FakeCuda(5, 2, 64), FakeCuda(5, 2, 64))
