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


def test_a_binding_that_does_not_load_says_why(monkeypatch, tmp_path):
    from paged_kv_cache_190_gb300 import _lib
    bad = tmp_path / "_step.so"
    bad.write_bytes(b"no library")
    monkeypatch.setattr(_lib, "_step", None)
    monkeypatch.setattr(_build, "binding_path", lambda: str(bad))
    with pytest.raises(RuntimeError, match=f"does not load.*{bad}"):
        _lib._binding()
    assert _lib._step is None


def test_the_first_calls_of_two_threads_load_one_binding(monkeypatch):
    import threading
    from paged_kv_cache_190_gb300 import _lib
    monkeypatch.setattr(_lib, "_step", None)
    got = []
    threads = [threading.Thread(target=lambda: got.append(_lib._binding())) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 8 and len({id(m) for m in got}) == 1
