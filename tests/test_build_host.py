"""When build.py builds the library and the binding again.  No compiler runs: the commands are recorded."""

import importlib.util
import json
import os
import shutil
import subprocess
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """A copy of build.py beside up-to-date sources and products, and the list of commands it ran."""
    pkg = tmp_path / "exact_io_aware_90_b200"
    shutil.copytree(os.path.join(ROOT, "exact_io_aware_90_b200", "csrc"), pkg / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    shutil.copy(os.path.join(ROOT, "exact_io_aware_90_b200", "build.py"), pkg / "build.py")
    spec = importlib.util.spec_from_file_location("_fa_build_copy", pkg / "build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    ran = []

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(subprocess, "run", run)
    mod.build()
    mod.ran = ran
    return mod


def test_nothing_is_built_twice(build):
    assert build.ran == ["nvcc", "g++"]
    build.build()
    assert build.ran == ["nvcc", "g++"]


@pytest.mark.parametrize("change", ["torch", "git", "cuda", "abi", "python", "record"])
def test_binding_follows_the_interpreter_and_torch(build, monkeypatch, change):
    import torch
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif change == "git":
        monkeypatch.setattr(torch.version, "git_version", "0000")
    elif change == "cuda":
        monkeypatch.setattr(torch.version, "cuda", "0.1")
    elif change == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    elif change == "python":
        monkeypatch.setattr(sys, "version", "0.0")
    else:
        os.remove(build.BUILT_FOR_PATH)
    build.build()
    assert build.ran == ["nvcc", "g++", "g++"]
    build.build()
    assert build.ran == ["nvcc", "g++", "g++"]
    with open(build.BUILT_FOR_PATH) as f:
        assert json.load(f)["torch"] == str(torch.__version__)


def test_sources_newer_than_their_product(build):
    late = os.path.getmtime(build.LIB_PATH) + 10
    os.utime(os.path.join(build.CSRC, "binding.cpp"), (late, late))
    build.build()
    assert build.ran == ["nvcc", "g++", "g++"]
    os.utime(os.path.join(build.CSRC, "fa_rope.cu"), (late, late))
    build.build()
    assert build.ran[3] == "nvcc"


def test_library_alone_without_torch(build, monkeypatch, capsys):
    """The C ABI needs no torch: without it the library is built, and the binding is left out with a word."""
    monkeypatch.setitem(sys.modules, "torch", None)
    os.remove(build.LIB_PATH)
    assert build.build() == build.LIB_PATH and build.ran[2:] == ["nvcc"]
    assert "torch" in capsys.readouterr().err
    assert build.build(force=True) == build.LIB_PATH and build.ran[3:] == ["nvcc"]
