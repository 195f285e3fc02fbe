"""The build's two parts (CPU): the C library, and the binding that the gated
delta rule's Python calls go through."""

import os
import sysconfig

import pytest
import torch

from kernelized_linear_attention_kata_b200 import _lib as L
from kernelized_linear_attention_kata_b200 import build as kbuild


def test_the_library_does_not_need_the_binding(monkeypatch):
    """It is built first, and a binding that cannot be built is a warning."""
    built = []

    def no_binding(force=False, verbose=False):
        built.append("binding")
        raise RuntimeError("Python.h: No such file or directory")
    real = kbuild.build_library
    monkeypatch.setattr(kbuild, "build_library", lambda *a: built.append("library") or real(*a))
    monkeypatch.setattr(kbuild, "build_binding", no_binding)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        path = kbuild.build()
    assert built == ["library", "binding"]
    assert path == kbuild.LIB_PATH and os.path.exists(path)


@pytest.mark.parametrize("error", [ImportError("No module named 'torch'"), FileNotFoundError("g++")])
def test_what_the_binding_lacks_is_told(monkeypatch, error):
    def no_binding(force=False, verbose=False):
        raise error
    monkeypatch.setattr(kbuild, "build_binding", no_binding)
    with pytest.warns(RuntimeWarning, match="gated delta rule"):
        kbuild.build()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    """Its name has torch's and Python's versions: after a change of either, the
    call says what is missing and the build makes it."""
    kbuild.build()
    here = kbuild.binding_path()
    assert os.path.exists(here) and sysconfig.get_config_var("EXT_SUFFIX") in here
    monkeypatch.setattr(torch, "__version__", "0.1.2+other")
    assert kbuild.binding_path() != here and not os.path.exists(kbuild.binding_path())
    monkeypatch.setattr(L, "_binding", None)
    with pytest.raises(ImportError, match="0.1.2"):
        L.binding()


def test_a_binding_that_does_not_load_says_why(monkeypatch, tmp_path):
    broken = tmp_path / "broken.so"
    broken.write_bytes(b"not a shared object")
    monkeypatch.setattr(kbuild, "binding_path", lambda: str(broken))
    monkeypatch.setattr(L, "_binding", None)
    kbuild.build_library()
    with pytest.raises(ImportError, match="(?s)broken.so.*--force"):
        L.binding()
