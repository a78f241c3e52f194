"""The build without a GPU: the C library needs nvcc and g++, its Python binding torch and
Python's headers as well."""
import os
import sys
import sysconfig

import pytest

from paged_kv_cache_190_gb300 import _build


@pytest.fixture
def only_the_binding(monkeypatch):
    """A build that finds everything up to date but the binding; its commands."""
    ran = []
    monkeypatch.setattr(_build, "_newer", lambda target, deps: "step" in os.path.basename(target))

    def run(cmd, **kw):
        ran.append(cmd)
        raise AssertionError(f"ran {cmd[:3]}")

    monkeypatch.setattr(_build.subprocess, "run", run)
    return ran


def test_the_library_builds_without_torch(monkeypatch, only_the_binding, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)               # import torch: ImportError
    assert _build.build() == _build.LIB
    assert not only_the_binding and "torch" in capsys.readouterr().err


def test_the_library_builds_without_python_headers(monkeypatch, only_the_binding, tmp_path, capsys):
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    assert _build.build() == _build.LIB
    assert not only_the_binding and "Python.h" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_is_an_error(monkeypatch, only_the_binding):
    with pytest.raises(AssertionError):
        _build.build()


def test_a_binding_belongs_to_one_torch_and_one_interpreter(monkeypatch):
    """A torch or a Python that was changed finds no binding made for another one."""
    import torch
    from paged_kv_cache_190_gb300 import _lib
    here = _build.binding_path()
    assert os.path.exists(here) and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(_lib, "_step", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert _build.binding_path() != here
    with pytest.raises(RuntimeError, match="0.0.1.other"):
        _lib._binding()
    monkeypatch.undo()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-other.so")
    assert _build.binding_path() != here
