"""The build's two parts (CPU): the C library, and the binding that the gated
delta rule's Python calls go through."""

import os

import pytest

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
