"""The library's build where there is no torch, or no g++: libgdn.so needs hipcc
alone, the Python extension a torch to bind and any C++ compiler."""
import os
import subprocess
import sys

import pytest

from speculative_verify_gdn_amd import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The build with its commands recorded instead of run, into an empty folder."""
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return seen


def test_with_torch(commands, monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", "some-c++")
    assert build.build() == str(tmp_path / "libgdn.so")
    assert commands[-1][0] == "some-c++" and (tmp_path / "_gdn_binding.so").exists()


@pytest.mark.parametrize("verbose", [False, True])
def test_without_torch(commands, monkeypatch, tmp_path, verbose, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)          # import torch raises ImportError
    assert build.build(verbose=verbose) == str(tmp_path / "libgdn.so")
    assert (tmp_path / "libgdn.so").exists() and not (tmp_path / "_gdn_binding.so").exists()
    assert all(c[0] == build.HIPCC for c in commands)
    assert ("no torch" in capsys.readouterr().out) == verbose


def test_without_a_host_compiler(commands, monkeypatch):
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    build.build_binding()
    assert commands[-1][:3] == [build.HIPCC, "-x", "c++"]


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not installed")
def test_the_rocm_compiler_builds_it(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert os.path.getsize(build.build_binding()) > 10000
