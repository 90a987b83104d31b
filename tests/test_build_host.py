"""What the build makes anew, on a copy of the outputs' names: the compilers are
stood in for by a function that writes the files that they were asked for."""
import os
import subprocess
import types

import pytest

from transformer_encoder_forward_gb300 import build as tebuild


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Runs a build with outputs in tmp_path; returns the base names of what was made."""
    monkeypatch.setattr(tebuild, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(tebuild, "LIB", str(tmp_path / "libtefwd.so"))
    monkeypatch.setattr(tebuild, "MARSHAL", str(tmp_path / "_marshal.so"))
    log = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        log.append(os.path.basename(out))
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)

    def go():
        log.clear()
        tebuild.build()
        return set(log)
    return go


MODULE = {"marshal.o", "_marshal.so.tmp"}


def test_everything_once(made):
    first = made()
    assert MODULE < first and "libtefwd.so.tmp" in first and "i8_linear.o" in first
    assert made() == set()


def test_another_torch_makes_the_module_anew(made, monkeypatch):
    import torch
    made()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert made() == MODULE
    assert made() == set()


def test_the_library_is_built_without_torch(made, monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "torch", None)          # an import of it fails
    first = made()
    assert "libtefwd.so.tmp" in first and not first & MODULE
    assert made() == set()
