"""What is built and loaded, and what is said where a part cannot be.  The compilers are replaced: nothing is compiled."""

import os
import subprocess
import types

import pytest
import torch

import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import build


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Outputs in a folder of the test's own; ``broken`` names the part whose compiler fails; ``ran`` what was built."""
    state = types.SimpleNamespace(ran=[], broken=None, lib=str(tmp_path / "libwmtp.so"), binding=str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "LIB", state.lib)
    monkeypatch.setattr(build._lib, "binding_path", lambda: state.binding)

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        part = "library" if out.startswith(state.lib) else "binding"
        state.ran.append(part)
        if part == state.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", run)
    return state


def test_library_is_built_where_the_binding_cannot_be(compilers):
    compilers.broken = "binding"
    with pytest.warns(UserWarning, match="step calls"):
        assert build.build() == compilers.lib
    assert os.path.exists(compilers.lib) and not os.path.exists(compilers.binding)
    with pytest.warns(UserWarning, match="no such header"):
        build.build()
    assert compilers.ran == ["library", "binding", "binding"]


def test_library_is_built_without_a_host_compiler_or_pytorch(compilers, monkeypatch):
    def missing(out):
        raise FileNotFoundError("g++")
    monkeypatch.setattr(build, "_build_binding", missing)
    with pytest.warns(UserWarning, match="step calls"):
        assert build.build() == compilers.lib
    assert compilers.ran == ["library"]


def test_a_library_that_cannot_be_built_is_an_error(compilers):
    compilers.broken = "library"
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()


def test_only_what_is_older_than_its_sources_is_built(compilers):
    build.build()
    build.build()
    assert sorted(compilers.ran) == ["binding", "library"]
    os.utime(compilers.binding, (0, 0))
    build.build()
    assert sorted(compilers.ran) == ["binding", "binding", "library"]
    build.build(force=True)
    assert sorted(compilers.ran) == ["binding"] * 3 + ["library"] * 2


def test_a_binding_for_another_pytorch_is_not_up_to_date(compilers, monkeypatch):
    monkeypatch.undo()  # the real names
    mine = build._lib.binding_path()
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    other = build._lib.binding_path()
    assert other != mine and "1.0.0+other" in other and not build.up_to_date(other)
    monkeypatch.setattr(build._lib.sysconfig, "get_config_var", lambda name: ".cpython-999.so")
    assert build._lib.binding_path().endswith(".cpython-999.so")


def _call():
    w.token_logprobs(torch.zeros(1, 8), torch.zeros(1, 1, dtype=torch.int32))


def test_step_calls_say_whether_the_binding_is_missing_or_broken(tmp_path, monkeypatch):
    build.build()
    path = tmp_path / "_step_binding.so"
    monkeypatch.setattr(w.step, "_native", None)
    monkeypatch.setattr(build._lib, "binding_path", lambda: str(path))
    with pytest.raises(ImportError, match="not found; build it"):
        _call()
    path.write_bytes(b"no library")
    with pytest.raises(ImportError) as e:  # the loader's own words
        _call()
    assert "not found" not in str(e.value) and "_step_binding" in str(e.value)
    monkeypatch.undo()
    with pytest.raises(ValueError, match="CUDA"):
        _call()
