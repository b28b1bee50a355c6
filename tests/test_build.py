"""When the library counts as out of date and what a failing part of the build leaves behind; the
compilers are stand-ins that only write their output file."""
import os
import subprocess
import types

import pytest

from test_neural_memory_gb300 import _build


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A library folder of its own, with compilers that succeed unless `fails` names the output."""
    fails = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        if any(f in out for f in fails):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        with open(out, "w") as f:
            f.write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(_build, "LIBDIR", str(tmp_path))
    for name in ("LIB", "BIND", "BIND_FOR"):
        if hasattr(_build, name):
            monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    return fails


def test_up_to_date_after_a_build(place):
    assert _build._stale()
    assert _build.build() == _build.LIB and os.path.exists(_build.BIND)
    assert not _build._stale()


@pytest.mark.parametrize("what", ["version", "SOABI"])
def test_another_torch_or_python_is_out_of_date(place, monkeypatch, what):
    import importlib.metadata
    import sysconfig
    _build.build()
    if what == "version":
        monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1")
    else:
        get = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-00" if n == "SOABI" else get(n))
    assert _build._stale()
    _build.build()
    assert not _build._stale()


@pytest.mark.parametrize("part", ["bind_train.cpp.o", "ttm_torch.so"])
def test_a_binding_that_fails_leaves_the_library(place, part):
    place.append(part)
    with pytest.raises(RuntimeError):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BIND) and _build._stale()
    place.clear()
    _build.build()
    assert not _build._stale()


def test_no_torch_builds_the_library_alone(place, monkeypatch):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    with pytest.raises(RuntimeError, match="torch"):
        _build.build()
    assert os.path.exists(_build.LIB)
