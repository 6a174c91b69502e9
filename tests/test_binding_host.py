"""The compiled calls (csrc/binding.cpp) without a GPU: an extension that does not fit this
torch or Python, and its build."""
import importlib
import os
import subprocess
import sys
import types

import pytest
import torch

PKG = "mixture_experts_expert_route_b200"


@pytest.fixture
def L():
    from mixture_experts_expert_route_b200 import _lib, build
    build.build()
    _lib.lib()
    return _lib


class Finder:
    """Loads the extension as `module`, or fails to with `error`."""

    def __init__(self, module=None, error=None):
        self.module, self.error = module, error

    def find_spec(self, name, path=None, target=None):
        if name != PKG + "._binding":
            return None
        if self.error:
            raise self.error
        return importlib.machinery.ModuleSpec(name, self)

    def create_module(self, spec):
        return self.module

    def exec_module(self, module):
        pass


@pytest.fixture
def extension(monkeypatch):
    """extension(finder): the next import of the extension asks that finder first."""
    pkg, name = importlib.import_module(PKG), PKG + "._binding"
    module, attribute = sys.modules.pop(name, None), pkg.__dict__.pop("_binding", None)
    yield lambda finder: monkeypatch.setattr(sys, "meta_path", [finder, *sys.meta_path])
    sys.modules.pop(name, None)
    pkg.__dict__.pop("_binding", None)
    if module is not None:
        sys.modules[name] = module
    if attribute is not None:
        pkg._binding = attribute


def test_an_extension_that_does_not_load_is_not_used(L, extension):
    """An undefined symbol, say: a warning, and the calls go through ctypes."""
    extension(Finder(error=ImportError("undefined symbol: _ZN2at")))
    calls = L._Calls()
    with pytest.warns(UserWarning, match="undefined symbol"):
        assert calls.linear(*range(9)) is NotImplemented
    assert calls.decode(*range(14)) is NotImplemented      # (bound: no second warning)


def test_an_extension_of_another_torch_is_not_used(L, extension):
    other = types.ModuleType(PKG + "._binding")
    other.torch_version = "1.0.0"
    other.init = lambda *a: pytest.fail("initialised")
    other.linear = other.decode = lambda *a: pytest.fail("called")
    extension(Finder(module=other))
    calls = L._Calls()
    with pytest.warns(UserWarning, match="torch 1.0.0"):
        assert calls.linear(*range(9)) is NotImplemented
    assert calls.decode(*range(14)) is NotImplemented


def test_no_extension_is_no_error(L, extension):
    extension(Finder(error=ModuleNotFoundError("_binding")))
    assert L._Calls().linear(*range(9)) is NotImplemented


def test_the_built_extension_fits(L):
    b = importlib.import_module(PKG + "._binding")
    assert b.torch_version == torch.__version__.split("+")[0]


def test_a_missing_library_stays_an_error(L, monkeypatch, tmp_path):
    monkeypatch.setattr(L, "LIB_PATH", str(tmp_path / "absent.so"))
    monkeypatch.setattr(L, "_lib", None)
    with pytest.raises(ImportError, match="absent.so"):
        L._Calls().linear(*range(9))


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """build.py with the extension's place in an empty folder, and the commands it runs."""
    from mixture_experts_expert_route_b200 import build
    commands = []

    def run(cmd):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "b" / "binding.txt"), raising=False)
    monkeypatch.setattr(build.subprocess, "check_call", run)
    return build, commands


def test_another_torch_rebuilds_the_extension(elsewhere, monkeypatch):
    build, commands = elsewhere
    build.build_binding()
    build.build_binding()
    assert len(commands) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_binding()
    build.build_binding()
    assert len(commands) == 2
    monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-399")
    build.build_binding()
    assert len(commands) == 3


@pytest.mark.parametrize("error", [FileNotFoundError("g++"),
                                   subprocess.CalledProcessError(1, ["g++"])])
def test_a_machine_that_cannot_build_the_extension(elsewhere, monkeypatch, error):
    """No compiler, or no headers: a warning, and no extension of other sources is left over."""
    build, commands = elsewhere
    build.build_binding()

    def run(cmd):
        raise error

    monkeypatch.setattr(build.subprocess, "check_call", run)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.warns(UserWarning, match="calls go through ctypes"):
        build.build_binding()
    assert not os.path.exists(build.BINDING)
