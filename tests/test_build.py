"""What a build runs: the compiler's calls are replaced by a record of them."""

import os
import shutil
import subprocess
import sys

import pytest

from sparsified_gradient_compression_amd import build as b


@pytest.fixture
def calls(monkeypatch, tmp_path):
    made = []

    def check_call(cmd):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(subprocess, "check_call", check_call)
    for name in ("LIB", "BINDING"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path))
    return made


def test_the_library_needs_hipcc_alone(calls, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    open(b.BINDING, "w").close()
    assert b.build(verbose=False) == b.LIB
    assert len(calls) == len(b.SOURCES) + 1 and all("hipcc" in c[0] for c in calls)
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)  # none of an earlier library
    assert not b.is_stale()


def test_the_torch_module_is_built_where_it_can_be(calls, monkeypatch):
    assert b.build(verbose=False) == b.LIB
    assert [c[0] for c in calls].count("g++") == 1 and os.path.exists(b.BINDING) and not b.is_stale()
    os.remove(b.BINDING)
    assert b.is_stale()
    monkeypatch.setattr(shutil, "which", lambda name: None)
    assert not b.is_stale()
