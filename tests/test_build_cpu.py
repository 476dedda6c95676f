"""What the build needs and when it builds the Python binding again (no compiler is run)."""
from __future__ import annotations

import importlib.metadata
import os
import subprocess
import sys
import types

import pytest

from softmax_learned_covariance_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A finished tree of its own: the library and its objects are newer than every source."""
    objs = tmp_path / "_build"
    objs.mkdir()
    for name in os.listdir(build.CSRC):
        if name.endswith(".cu"):
            (objs / (name[:-3] + ".o")).write_bytes(b"")
    for name in ("libparallax.so", "_binding.so"):
        (tmp_path / name).write_bytes(b"")
    monkeypatch.setattr(build, "BUILD", str(objs))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libparallax.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(subprocess, "check_call", lambda cmd, **kw: run(cmd))
    return tmp_path, ran


def test_the_library_is_built_without_torch(tree, monkeypatch):
    path, ran = tree
    os.remove(path / "libparallax.so")
    os.remove(path / "_binding.so")
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == str(path / "libparallax.so")
    assert os.path.exists(path / "libparallax.so") and not os.path.exists(path / "_binding.so")
    assert len(ran) == 1                                 # the link


def test_the_binding_is_built_again_for_another_torch(tree, monkeypatch):
    path, ran = tree
    build.build()
    n = len(ran)
    build.build()
    assert len(ran) == n                                 # nothing to do
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1" if name == "torch" else real(name))
    build.build()
    assert len(ran) == n + 1 and any(str(a).endswith("binding.cpp") for a in ran[-1])
    build.build()
    assert len(ran) == n + 1
