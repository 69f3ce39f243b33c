"""What build() runs, with the compilers' calls recorded instead of made.  No GPU."""

import importlib
import importlib.util

import pytest

b = importlib.import_module("flow_matching_dit_b200.build")   # (the package's attribute of this name is the function)


@pytest.fixture
def runs(monkeypatch):
    """The outputs that build() would compile, in order."""
    made = []
    monkeypatch.setattr(b, "_run", lambda cmd, tmp, out, verbose: made.append(out))
    return made


def test_the_checked_library_needs_neither_torch_nor_the_binding(runs, monkeypatch):
    def no_binding(*_):
        raise AssertionError("the binding is not part of the checked library")
    monkeypatch.setattr(b, "binding_command", no_binding)
    assert b.build(force=True, checked=True) == b.LIB_CHECKED
    assert runs == [b.LIB_CHECKED]


def test_the_library_is_built_without_torch(runs, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert b.build(force=True) == b.LIB
    assert runs == [b.LIB] and "not built" in capsys.readouterr().err


def test_the_library_and_the_binding(runs, monkeypatch):
    assert b.build(force=True) == b.LIB
    assert runs == [b.LIB, b.BINDING]
    del runs[:]
    monkeypatch.setattr(b, "up_to_date", lambda lib: True)
    monkeypatch.setattr(b, "binding_up_to_date", lambda: True)
    assert b.build() == b.LIB and runs == []
