"""The compiled binding belongs to one interpreter and one torch: another finds none and builds its own."""

import sysconfig
from importlib import metadata

from ragged_log_probs_gb300 import _build


def test_binding_is_named_after_its_interpreter_and_torch(monkeypatch):
    here = _build.binding_path()
    _build.build()
    assert _build.up_to_date()
    monkeypatch.setattr(metadata, "version", lambda name: "0.0.1")
    assert _build.binding_path() != here and not _build.up_to_date()
    monkeypatch.undo()
    assert _build.binding_path() == here and _build.up_to_date()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-none")
    assert _build.binding_path() != here and not _build.up_to_date()
