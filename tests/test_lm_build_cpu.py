"""What building the library needs: nvcc alone for the C library and its test-only variants, torch
and a C++ compiler for the Python binding of the operators around the FFN, which is built again for
another Python or torch.  (The compilers are stand-ins that write empty files.)"""
import importlib.util
import os
import subprocess

import pytest

from activation_sparse_transformer_gate_gb300 import _build


@pytest.fixture
def calls(monkeypatch, tmp_path):
    got = []

    def run(cmd, **kw):
        got.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    monkeypatch.setattr(_build, "OBJDIR", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_lm.so"))
    if hasattr(_build, "STAMP"):
        monkeypatch.setattr(_build, "STAMP", str(tmp_path / "objects" / "lib" / "lm_bind.for"))
    monkeypatch.setattr(_build, "nvcc_path", lambda: "nvcc")
    monkeypatch.setattr(subprocess, "run", run)
    return got


def hide_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_without_torch(calls, monkeypatch, tmp_path, capsys):
    hide_torch(monkeypatch)
    lib = _build.build()
    assert os.path.exists(lib) and {c[0] for c in calls} == {"nvcc"}
    assert not os.path.exists(_build.BINDING)
    assert "no Python binding" in capsys.readouterr().err
    calls.clear()
    _build.build()
    assert not calls                                   # nothing to do a second time


def test_test_variants_without_torch(calls, monkeypatch):
    hide_torch(monkeypatch)
    lib = _build.build(variants=("hooks", "timeout"))
    assert os.path.exists(lib) and {c[0] for c in calls} == {"nvcc"}


def test_binding_goes_by_python_and_torch(calls, monkeypatch):
    _build.build()
    assert os.path.exists(_build.BINDING) and "g++" in {c[0] for c in calls}
    calls.clear()
    _build.build()
    assert not calls
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-999")
    _build.build()
    assert "g++" in {c[0] for c in calls}
