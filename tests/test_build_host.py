"""Building the library and loading the binding's compiled checks (no GPU): the
library needs nothing of the checks, and checks of another torch are not used."""

import os
import subprocess
import sys
import types

import pytest

import all_reduce_reduction_rank_amd as ar
from all_reduce_reduction_rank_amd import binding, build

NAME = ar.__name__ + "._marshal"


@pytest.mark.parametrize("error", [RuntimeError("g++ failed on marshal.cpp"), FileNotFoundError("g++"), ImportError("no torch")])
def test_library_builds_without_the_checks(tmp_path, monkeypatch, capsys, error):
    def compiler(cmd, **kw):  # leaves its output, as hipcc does
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def fails(out=None):
        raise error

    lib, marshal = tmp_path / "libar.so", tmp_path / "_marshal.so"
    marshal.write_text("of an earlier build")
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "MARSHAL", str(marshal))
    monkeypatch.setattr(build, "build_marshal", fails)
    monkeypatch.setattr(build.subprocess, "run", compiler)
    assert build.build(out=str(lib)) == str(lib)
    assert lib.exists() and not marshal.exists()  # what was there may not fit the binding
    assert str(error) in capsys.readouterr().err


def _reload(monkeypatch):
    monkeypatch.setattr(binding, "_TORCH", None)
    monkeypatch.setattr(binding, "_MARSHAL", None)
    binding._torch()
    return binding._MARSHAL


def test_checks_that_were_built_are_loaded(monkeypatch):
    if not os.path.exists(build.MARSHAL):
        pytest.skip("built with the library")
    found = _reload(monkeypatch)
    assert found is not None and found.BUILT_FOR == build.checks_built_for()


def test_checks_of_another_torch_are_not_used(monkeypatch):
    for other in (types.SimpleNamespace(BUILT_FOR="torch 1.0, python 3.10"), types.SimpleNamespace()):
        monkeypatch.setitem(sys.modules, NAME, other)
        with pytest.warns(RuntimeWarning, match="_marshal.so was built for"):
            assert _reload(monkeypatch) is None


def test_checks_that_do_not_load_are_named(monkeypatch, tmp_path):
    bad = tmp_path / "_marshal.so"
    bad.write_text("no library")
    monkeypatch.delitem(sys.modules, NAME, raising=False)
    monkeypatch.setattr(ar, "__path__", [str(tmp_path)])
    with pytest.warns(RuntimeWarning, match="_marshal.so does not load"):
        assert _reload(monkeypatch) is None


def test_without_checks_nothing_is_said(monkeypatch, tmp_path, recwarn):
    monkeypatch.delitem(sys.modules, NAME, raising=False)
    monkeypatch.setattr(ar, "__path__", [str(tmp_path)])
    assert _reload(monkeypatch) is None and not recwarn.list
