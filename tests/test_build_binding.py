"""The build goes through without the compiled binding, whose calls the ctypes functions then make (no GPU)."""
import importlib.util
import os

import pytest
import torch  # noqa: F401

from ragged_grouped_gemm_device_gb300 import build


def test_without_torch(monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert build.build_binding(force=True) is None


@pytest.mark.parametrize("cause", ["compile", "compiler", "headers"])
def test_without_an_extension(cause, monkeypatch, tmp_path, capfd):
    csrc, old = tmp_path / "csrc", tmp_path / "_binding.so"
    csrc.mkdir()
    (csrc / "binding.cpp").write_text("this does not compile\n")
    old.write_bytes(b"an extension of older sources")
    os.utime(old, (1, 1))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "BINDING", str(old))
    if cause == "compiler":
        real = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda c: None if c in ("g++", "c++") else real(c))
    if cause == "headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build_binding() is None
    assert not old.exists()  # it would be loaded in place of the ctypes functions
    assert ("does not compile" in capfd.readouterr().err) == (cause == "compile")
