"""What the build makes when a part of it cannot be made, and when a part is out of date."""
import os

import pytest
import torch

import exact_io_aware_08_gb300 as fa
from exact_io_aware_08_gb300 import build as fabuild


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build of one small source, outside the tree."""
    monkeypatch.setattr(fabuild, "LIB", str(tmp_path / "libfa.so"))
    monkeypatch.setattr(fabuild, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(fabuild, "_sources", lambda: [os.path.join(fabuild.CSRC, "selftest.cu")])
    return tmp_path


def test_the_library_is_made_without_the_module(elsewhere, monkeypatch):
    """Without torch's headers (or g++) the C ABI is built all the same, and the error still goes up."""
    def fails():
        raise RuntimeError("g++ failed for binding.cpp")
    monkeypatch.setattr(fabuild, "build_binding", fails)
    monkeypatch.setattr(fabuild, "binding_up_to_date", lambda: False)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        fabuild.build()
    assert (elsewhere / "libfa.so").exists()


def test_the_library_alone(elsewhere, monkeypatch):
    def wanted():
        pytest.fail("the module was asked for")
    monkeypatch.setattr(fabuild, "build_binding", wanted)
    monkeypatch.setattr(fabuild, "binding_up_to_date", wanted)
    assert fabuild.build(binding=False) == str(elsewhere / "libfa.so")
    assert fabuild.up_to_date()


def test_another_torch_finds_no_module(monkeypatch):
    """The module is made of one torch's C++ classes: with another it is out of date, and not loaded."""
    fabuild.build()
    assert fabuild.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert not fabuild.binding_up_to_date()
    monkeypatch.setattr(fa, "_native", None)
    with pytest.raises(fa.FaError, match="not found"):
        fa._binding()


def test_another_python_finds_no_module(monkeypatch):
    path = fabuild.binding_path()
    monkeypatch.setattr(fabuild.sys.implementation, "cache_tag", "cpython-999")
    assert fabuild.binding_path() != path and "cpython-999" in fabuild.binding_path()
