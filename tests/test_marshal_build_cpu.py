"""The binding's check in C is used only where it was built for this Python and this torch, and
nothing else depends on it."""

import sys
import sysconfig
import types

import pytest
import torch

import moe_decode_layer_router_amd as mb
from moe_decode_layer_router_amd import _build

NAME = "moe_decode_layer_router_amd._marshal"


def _python(*args):
    raise AssertionError("not called")


def _module(**kw):
    m = types.ModuleType(NAME)
    m.buf, m.set_python = (lambda *a: None), (lambda f: None)
    m.__dict__.update(kw)
    return m


@pytest.fixture
def loaded(monkeypatch):
    def put(m):
        monkeypatch.setitem(sys.modules, NAME, m)
        monkeypatch.setattr(mb, "_marshal", m, raising=False)

    return put


def test_of_this_torch(loaded):
    m = _module(torch_build=f"{torch.__version__} {torch.version.git_version}")
    loaded(m)
    assert mb._check_in_c(_python) is m.buf


@pytest.mark.parametrize("kw", [{}, dict(torch_build="2.1.0 0123"), dict(torch_build=torch.__version__)])
def test_of_another_torch(loaded, kw):
    loaded(_module(**kw))
    assert mb._check_in_c(_python) is _python


def test_its_name_is_of_this_python():
    assert _build.MARSHAL.endswith("_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("cxx", ["false", "no-such-compiler"])
def test_without_a_compiler(monkeypatch, tmp_path, capsys, cxx):
    """No error, and no older file is left to be loaded."""
    old = tmp_path / ("_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
    any_python = tmp_path / "_marshal.so"
    for f in (old, any_python):
        f.write_bytes(b"older")
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    monkeypatch.setattr(_build, "MARSHAL", str(old))
    monkeypatch.setenv("CXX", cxx)
    assert _build.build_marshal() is None
    assert not old.exists() and not any_python.exists()
    assert "the one in Python serves" in capsys.readouterr().err
