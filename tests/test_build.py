"""The build: the C library needs no PyTorch, and the Python entries fit the one that they were compiled against."""
import importlib.metadata
import os
import sys

import pytest

from mixture_experts_layer_gate_gb300 import build


@pytest.fixture
def small(monkeypatch, tmp_path):
    """A build of one source into an empty directory."""
    monkeypatch.setattr(build, "SOURCES", ["repack.cu"])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoe_gb300.so"))
    monkeypatch.setattr(build, "OPS", str(tmp_path / "_ops.so"))


def test_library_without_pytorch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.OPS)


def test_library_is_there_when_the_python_entries_fail(small, monkeypatch):
    monkeypatch.setattr(build, "_ops_command", lambda obj: ["false"])
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.OPS)


def test_python_entries_are_built_again_for_another_pytorch(small, monkeypatch):
    ran = []
    monkeypatch.setattr(build, "_ops_command", lambda obj: (ran.append("compile"), ["touch", obj])[1])
    monkeypatch.setattr(build, "_link_ops", lambda obj: (ran.append("link"), ["cp", obj, build.OPS])[1])
    build.build()
    assert ran == ["compile", "link"]
    build.build()
    assert ran == ["compile", "link"]
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0" if name == "torch" else version(name))
    build.build()
    assert ran == ["compile", "link"] * 2
    monkeypatch.setattr(importlib.metadata, "version", version)
    build.build()                                 # back: the object is there, the entries are not of it
    assert ran == ["compile", "link"] * 2 + ["link"]
