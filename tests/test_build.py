"""What the build makes, and when (compilers replaced by stand-ins)."""
import builtins
import os
import subprocess
import types
from importlib import metadata

import pytest

from activation_sparse_decode_threshold_b200 import build as b


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """A build into a folder of its own, whose compilers only write their outputs; the outputs' names in order."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        made.append(os.path.basename(out))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "subprocess", types.SimpleNamespace(run=run))
    for name, path in (("OUT", "lib.so"), ("EXT", "ext.so"), ("OBJ", "obj"), ("EXT_FOR", "ext.for")):
        monkeypatch.setattr(b, name, str(tmp_path / path), raising=False)   # (the last is newer than the others)
    return made


def test_the_library_is_built_without_torch(commands, monkeypatch):
    real = builtins.__import__

    def no_torch(name, *a, **kw):
        if name.split(".")[0] == "torch":
            raise ImportError("no torch here")
        return real(name, *a, **kw)

    def no_version(name):
        raise metadata.PackageNotFoundError(name)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    monkeypatch.setattr(metadata, "version", no_version)
    assert b.build() == b.OUT and os.path.exists(b.OUT) and not os.path.exists(b.EXT)
    assert not any("ext" in c for c in commands)


def test_a_second_build_does_nothing(commands):
    b.build()
    assert "lib.so.tmp" in commands and "ext.so.tmp" in commands and len(commands) == len(b.SOURCES) + 2
    commands.clear()
    b.build()
    assert commands == []


def test_the_native_part_follows_torch_s_version(commands, monkeypatch):
    b.build()
    commands.clear()
    monkeypatch.setattr(metadata, "version", lambda name: "9.9.9+other")
    b.build()
    assert commands == ["ext.so.tmp"]
    b.build()
    assert commands == ["ext.so.tmp"]


def test_a_native_part_that_fails_leaves_the_library(commands, monkeypatch):
    run = b.subprocess.run

    def failing(cmd, **kw):
        return subprocess.CompletedProcess(cmd, 1, "", "no headers") if cmd[0] == "g++" else run(cmd, **kw)

    monkeypatch.setattr(b, "subprocess", types.SimpleNamespace(run=failing))
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        b.build()
    assert os.path.exists(b.OUT)
