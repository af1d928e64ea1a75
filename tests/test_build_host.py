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
