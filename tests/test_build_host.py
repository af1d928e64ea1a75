"""The in-tree build: what counts as built, and what it does without the headers of the Python module."""
import os
import sysconfig

import pytest
import torch

from linear_recurrent_rnn_gb300 import build as B_
from linear_recurrent_rnn_gb300 import librglru as R


def test_a_module_for_another_torch_or_python_is_not_this_one(monkeypatch):
    B_.build()
    assert not B_.stale() and B_.binding_path() == B_.BINDING and os.path.exists(B_.BINDING)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.9.1+other")
        assert B_.binding_path() != B_.BINDING
        m.setattr(B_, "BINDING", B_.binding_path())
        assert B_.stale()
        m.setattr(R, "_calls", None)
        with pytest.raises(RuntimeError, match="not built"):
            R._paged_calls()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other")
        assert B_.binding_path() != B_.BINDING


@pytest.fixture
def small(monkeypatch, tmp_path):
    """The build of one source file in a folder of its own."""
    monkeypatch.setattr(B_, "SOURCES", ["host_util.cu"])
    monkeypatch.setattr(B_, "BUILD", str(tmp_path))
    monkeypatch.setattr(B_, "LIB", str(tmp_path / "librglru.so"))
    monkeypatch.setattr(B_, "BINDING", str(tmp_path / "rglru_binding.so"))
    return monkeypatch


def test_without_python_s_headers_the_library_is_built(small, capsys):
    paths = dict(sysconfig.get_paths(), include="/nowhere")
    small.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    assert B_.build() == B_.LIB and os.path.exists(B_.LIB)
    assert "/nowhere/Python.h" in capsys.readouterr().err
    assert not os.path.exists(B_.BINDING) and not B_.stale()
    small.setattr(R, "_calls", None)
    with pytest.raises(RuntimeError, match="not built"):
        R._paged_calls()


def test_a_module_that_does_not_compile_leaves_the_library(small, tmp_path):
    """An error of the module is raised, and the library is there."""
    small.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    (tmp_path / "Python.h").write_text("#error not Python's\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B_.build()
    assert os.path.exists(B_.LIB) and not os.path.exists(B_.BINDING) and B_.stale()
