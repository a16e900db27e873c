"""When the marshalling module is compiled again (nothing is compiled here)."""
import importlib.metadata
import os
import subprocess
import types

import pytest

from block_sparse_full_b200 import build as b


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """_build_marshal with a compiler that only writes its output; the commands it was given."""
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("so")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(subprocess, "run", run)
    return calls


def test_marshal_follows_torch_and_python(compiled, monkeypatch):
    b._build_marshal(False, False)
    assert len(compiled) == 1
    b._build_marshal(False, False)
    assert len(compiled) == 1  # nothing has changed
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda n: "99.0" if n == "torch" else version(n))
    b._build_marshal(False, False)
    assert len(compiled) == 2
    b._build_marshal(False, False)
    assert len(compiled) == 2
    monkeypatch.setattr(b.sys.implementation, "cache_tag", "cpython-999")
    b._build_marshal(False, False)
    assert len(compiled) == 3


def test_marshal_follows_its_sources(compiled):
    b._build_marshal(False, False)
    os.utime(b.MARSHAL, (1, 1))
    b._build_marshal(False, False)
    assert len(compiled) == 2
    b._build_marshal(False, True)
    assert len(compiled) == 3


def test_a_failed_compilation_is_tried_again(compiled, monkeypatch):
    good = subprocess.run
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no"))
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        b._build_marshal(False, False)
    monkeypatch.setattr(subprocess, "run", good)
    b._build_marshal(False, False)
    assert len(compiled) == 1 and os.path.exists(b.MARSHAL)


def test_the_library_is_built_without_torch(compiled, monkeypatch, capsys):
    # libssa.so is for C programs too: nothing but its own binding needs torch
    find = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    b._build_marshal(False, False)
    assert not compiled and "torch" in capsys.readouterr().out
