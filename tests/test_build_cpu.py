"""The build of the binding's extension module: when it is made again, and what a
call says where it cannot be used (a stand-in for the compiler; nothing is built)."""

import os
import stat

import pytest

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import _build
from load_balanced_paged_assign_gb300 import binding as E


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """A module path of its own, and a compiler that writes a file and counts its runs."""
    log = tmp_path / "runs"
    cxx = tmp_path / "cxx"
    cxx.write_text(f'#!/bin/sh\necho run >> {log}\nwhile [ "$1" != -o ]; do shift; done\n'
                   'echo module > "$2"\n')
    cxx.chmod(cxx.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("CXX", str(cxx))
    monkeypatch.setattr(_build, "EXT_PATH", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(_build, "EXT_STAMP", str(tmp_path / "_tensors.so.stamp"), raising=False)
    return lambda: log.read_text().count("run") if log.exists() else 0


def test_the_module_is_built_again_for_another_pytorch(compiler, monkeypatch):
    import torch
    _build.build_extension()
    _build.build_extension()
    assert compiler() == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    _build.build_extension()
    assert compiler() == 2
    _build.build_extension()
    assert compiler() == 2
    os.remove(_build.EXT_STAMP)  # one that does not say what it was built for
    _build.build_extension()
    assert compiler() == 3


def test_a_module_of_another_pytorch_is_not_loaded(compiler, monkeypatch):
    import torch
    _build.build_extension()
    monkeypatch.setattr(E, "_DENSE", None)

    def refused():
        with pytest.raises(RuntimeError, match="another PyTorch"):
            hd.hpc_decode_plan_win(torch.zeros(1, dtype=torch.int32), 1, 1, 1, 1, None)
        return E._DENSE is None

    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.9.9")
        assert refused()
    os.remove(_build.EXT_STAMP)
    assert refused()


def test_a_module_that_does_not_load_says_why(compiler, monkeypatch):
    import sys
    import torch
    package = hd.__name__
    monkeypatch.setattr(E, "_DENSE", None)
    monkeypatch.delattr(sys.modules[package], "_tensors", raising=False)

    class Broken:  # finds the module, and cannot load it
        @staticmethod
        def find_spec(name, path=None, target=None):
            if name == package + "._tensors":
                raise ImportError("undefined symbol: some_symbol")

    monkeypatch.delitem(sys.modules, package + "._tensors", raising=False)
    monkeypatch.setattr(sys, "meta_path", [Broken] + sys.meta_path)
    call = (torch.zeros(1, dtype=torch.int32), 1, 1, 1, 1, None)
    with pytest.raises(RuntimeError, match="is missing"):
        hd.hpc_decode_plan_win(*call)
    _build.build_extension()
    with pytest.raises(RuntimeError, match="undefined symbol: some_symbol"):
        hd.hpc_decode_plan_win(*call)


@pytest.mark.parametrize("without", ["compiler", "headers"])
def test_the_library_is_built_without_the_module(compiler, monkeypatch, without):
    """A caller of the C ABI needs nvcc only: no g++, or no PyTorch, is a warning."""
    made = []
    monkeypatch.setattr(_build, "is_stale", lambda: True)
    monkeypatch.setattr(_build, "_build_library", lambda *a: made.append(a[0]))
    if without == "compiler":
        monkeypatch.setenv("CXX", "/nonexistent/g++")
    else:
        import sys
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    with pytest.warns(UserWarning, match="_tensors was not built"):
        assert _build.build() == _build.LIB_PATH
    assert made == [_build.LIB_PATH] and not os.path.exists(_build.EXT_PATH)
    with pytest.raises((RuntimeError, OSError, ImportError)):
        _build.build_extension()
