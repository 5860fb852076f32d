"""When the Python module beside the library is built again: its sources, the PyTorch and the
Python that it is built for, or the flags have changed.  The compiler is a stand-in that
writes a file."""
import os
import sysconfig
import types

import pytest
import torch

from fp8_gemms_b200 import build


@pytest.fixture
def native(tmp_path, monkeypatch):
    """build_native into a folder of its own; .commands: what it ran."""
    out = types.SimpleNamespace(commands=[], path=str(tmp_path / "_native.so"))

    def run(cmd, check):
        out.commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
    monkeypatch.setattr(build, "NATIVE", out.path)
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    return out


def test_built_once(native):
    assert build.build_native() == native.path
    build.build_native()
    assert len(native.commands) == 1 and os.path.exists(native.path)
    build.build_native(force=True)
    assert len(native.commands) == 2


@pytest.mark.parametrize("change", ["torch", "torch source", "python", "c++ abi", "flags"])
def test_built_again_for_another(native, monkeypatch, change):
    build.build_native()
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    elif change == "torch source":
        monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    elif change == "python":
        was = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda n: "cpython-399-x86_64-linux-gnu" if n == "SOABI" else was(n))
    elif change == "c++ abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        monkeypatch.setattr(build, "NATIVE_FLAGS", ["-O3"], raising=False)
    build.build_native()
    build.build_native()
    assert len(native.commands) == 2


def test_not_built_again_where_the_tools_lie_elsewhere(native, monkeypatch):
    """A built tree runs on a machine of the same image with another environment."""
    build.build_native()
    monkeypatch.setenv("CXX", "/elsewhere/g++")
    monkeypatch.setenv("CUDA_HOME", "/elsewhere/cuda")
    build.build_native()
    assert len(native.commands) == 1


def test_built_again_after_a_build_that_failed(native, monkeypatch):
    """A module from before stays, but is not taken for one of the new kind."""
    build.build_native()
    good = build.subprocess

    def fails(cmd, check):
        raise RuntimeError("no compiler")
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=fails))
    with pytest.raises(RuntimeError):
        build.build_native()
    monkeypatch.setattr(build, "subprocess", good)
    build.build_native()
    assert len(native.commands) == 2


def test_built_again_when_a_source_is_newer(native, tmp_path, monkeypatch):
    source = tmp_path / "binding.cpp"
    source.write_text("")
    monkeypatch.setattr(build, "BINDING", str(source))
    build.build_native()
    late = os.path.getmtime(native.path) + 10
    os.utime(source, (late, late))
    build.build_native()
    assert len(native.commands) == 2
