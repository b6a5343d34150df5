"""The C library's build does not depend on the tensor binding's, and a missing binding is named."""
import builtins
import os
import shutil
import sys

import pytest

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import build as B
from sparse_long_context_gb300 import ops


@pytest.fixture
def fresh(lib, tmp_path, monkeypatch):
    """The build's outputs in a folder of their own (objects that exist already are taken over)."""
    objs = tmp_path / "objs"
    if os.path.isdir(B.BUILD):
        shutil.copytree(B.BUILD, objs)  # times are kept
    monkeypatch.setattr(B, "BUILD", str(objs))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsls.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    return tmp_path


def test_library_is_linked_without_gxx(fresh, monkeypatch):
    """Fails for want of g++ after the library, which a load then takes."""
    run = B.subprocess.run

    def no_gxx(cmd, **kw):
        if os.path.basename(cmd[0]) == "g++":
            raise FileNotFoundError(cmd[0])
        return run(cmd, **kw)

    monkeypatch.setattr(B.subprocess, "run", no_gxx)
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    os.remove(B.LIB)
    monkeypatch.setattr(L, "LIB_PATH", B.LIB)
    monkeypatch.setattr(L, "_lib", None)
    assert L.load(build_if_missing=True).sls_version() > 0


def test_library_is_linked_without_torch(fresh, monkeypatch):
    real = builtins.__import__

    def no_torch(name, *args, **kw):
        if name == "torch":
            raise ImportError(name)
        return real(name, *args, **kw)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    with pytest.raises(RuntimeError, match="needs torch"):
        B.build()
    assert os.path.exists(B.LIB)


def test_missing_binding_is_named(lib, monkeypatch):
    monkeypatch.setattr(ops, "_fast", None)
    name = ops.__name__.rsplit(".", 1)[0] + "._binding"
    monkeypatch.setitem(sys.modules, name, None)  # an import of it fails
    package = sys.modules[name.rsplit(".", 1)[0]]
    if hasattr(package, "_binding"):
        monkeypatch.delattr(package, "_binding")
    with pytest.raises(RuntimeError, match="tensor binding.*build it first"):
        ops._binding()
