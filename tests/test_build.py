"""The build (CPU only): the CUDA library needs nvcc alone; the extension module beside it needs torch,
a host compiler and Python's headers, and is left out where one is missing."""
import shutil
import sys
import sysconfig

import pytest

from recurrent_vision_backbone_b200 import build


@pytest.fixture
def lib(tmp_path, monkeypatch):
    """The CUDA library up to date, no extension module yet."""
    path = build.build()
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_ops.so"))
    return path


def test_extension_module(lib):
    assert build.build() == lib
    assert not build.is_stale(build.BINDING, build.BINDING_DEPS)


@pytest.mark.parametrize("missing", ["torch", "g++", "Python.h"])
def test_library_alone(lib, missing, monkeypatch, capfd, tmp_path):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)   # as if it were not installed
    elif missing == "g++":
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    else:
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    assert build.build() == lib
    assert missing in capfd.readouterr().err
    assert build.is_stale(build.BINDING, build.BINDING_DEPS)   # a later build makes it


def test_extension_module_of_another_torch(lib, monkeypatch):
    """The module is compiled against torch's headers: with another torch it is built anew."""
    import torch
    built = []
    monkeypatch.setattr(build, "binding_cmd", lambda out: built.append(out) or [sys.executable, "-c", f"open({out!r}, 'w')"])
    assert build.binding_is_stale()
    build.build()
    build.build()
    assert len(built) == 1 and not build.binding_is_stale()
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert build.binding_is_stale()
    build.build()
    assert len(built) == 2 and not build.binding_is_stale()
