"""The conveniences on torch tensors are compiled again for another torch or Python, and not loaded before."""
from __future__ import annotations

import subprocess

import pytest
import torch

from nvfp4_quantization_group_b200 import _build, layer


def test_conveniences_of_another_torch_are_stale(monkeypatch):
    _build.build_torch()
    assert _build.torch_lib_fits() and torch.__version__ in _build.built_for()
    compiled = []

    def run(cmd, **kw):
        compiled.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "not run")

    monkeypatch.setattr(_build.subprocess, "run", run)
    assert _build.build_torch() == _build.TORCH_LIB and not compiled
    real = _build.importlib.metadata.version
    monkeypatch.setattr(_build.importlib.metadata, "version", lambda n: "2.0.0" if n == "torch" else real(n))
    assert not _build.torch_lib_fits()
    with pytest.raises(RuntimeError, match="not run"):
        _build.build_torch()
    assert any("torch 2.0.0," in a for a in compiled[0])
    monkeypatch.setattr(layer, "_torch_calls", None)
    with pytest.raises(OSError, match="another torch"):
        layer._x()


def test_missing_conveniences_raise(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "TORCH_LIB", str(tmp_path / "none.so"))
    monkeypatch.setattr(layer, "_torch_calls", None)
    with pytest.raises(OSError, match="missing"):
        layer._x()
