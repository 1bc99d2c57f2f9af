"""The build's two parts, without a GPU: the C library needs nvcc alone, and the
Python binding's file belongs to one Python and one torch."""
import os
import sysconfig

import pytest
import torch

import integer_only_quantized_int8_b200 as ivit
from integer_only_quantized_int8_b200 import build as ivit_build


class Ran(Exception):
    pass


@pytest.fixture
def commands(monkeypatch):
    """Compilers that note their command lines and write the file that is asked for."""
    seen = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **_):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(ivit_build.subprocess, "run", run)
    return seen


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """Built files in a folder of their own."""
    monkeypatch.setattr(ivit_build, "LIB", str(tmp_path / "libivit_b200.so"))
    monkeypatch.setattr(ivit_build, "binding_path", lambda: str(tmp_path / "_binding.so"))
    return tmp_path


def test_library_needs_nothing_but_nvcc(commands, elsewhere, monkeypatch):
    def no_binding(*_):
        raise Ran

    monkeypatch.setattr(ivit_build, "build_binding", no_binding)
    assert ivit_build.build_library() == ivit_build.LIB
    assert os.path.exists(ivit_build.LIB)
    assert [os.path.basename(c[0]) for c in commands] == ["nvcc"]
    assert not any("torch" in a or "python" in a.lower() for a in commands[0])


def test_library_is_built_before_the_binding(commands, elsewhere, monkeypatch):
    """A missing g++, torch or Python header leaves a whole C library behind."""
    def no_binding(*_):
        assert os.path.exists(ivit_build.LIB)
        raise Ran

    monkeypatch.setattr(ivit_build, "build_binding", no_binding)
    with pytest.raises(Ran):
        ivit_build.build()


def test_binding_belongs_to_one_python_and_torch(monkeypatch):
    path = ivit_build.binding_path()
    name = os.path.basename(path)
    assert os.path.dirname(path) == os.path.dirname(ivit_build.LIB)
    assert name.startswith("_binding.") and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    other = ivit_build.binding_path()
    assert other != path
    monkeypatch.undo()
    monkeypatch.setattr(ivit_build.sysconfig, "get_config_var", lambda _: ".cpython-399-other.so")
    assert ivit_build.binding_path() not in (path, other)


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    """Under another torch the call names the build command; the file of this one stays untouched."""
    ivit_build.build()
    before = os.stat(ivit_build.binding_path())
    monkeypatch.setattr(ivit, "_calls", None)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    with pytest.raises(RuntimeError, match="native binding is missing"):
        ivit._native()
    monkeypatch.undo()
    assert os.stat(ivit_build.binding_path()) == before
    assert ivit._native() is not None


def test_binding_is_rebuilt_when_a_source_is_newer(commands, elsewhere):
    path = ivit_build.build_binding()
    assert len(commands) == 1
    newest = max(os.path.getmtime(p) for p in ivit_build.binding_deps())
    os.utime(path, (newest + 1, newest + 1))
    assert ivit_build.build_binding() == path and len(commands) == 1
    os.utime(path, (newest - 1, newest - 1))
    ivit_build.build_binding()
    assert len(commands) == 2
    ivit_build.build_binding(force=True)
    assert len(commands) == 3
