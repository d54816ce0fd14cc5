"""The binding's check of a tensor argument in C against the one in Python: the same pointers,
errors and messages."""

import importlib

import pytest
import torch

import moe_decode_layer_router_amd as mb

_marshal = pytest.importorskip("moe_decode_layer_router_amd._marshal", exc_type=ImportError)

F32, I32 = (torch.float32,), (torch.int32,)
T = torch.zeros((4, 4))


def _outcome(f, args):
    try:
        return f(*args)
    except Exception as e:
        return type(e), str(e)


def _python_buf():
    """_buf as the module defines it, before the first call puts the C one in its place."""
    spec = importlib.util.spec_from_file_location("moe_binding_fresh", mb.__file__, submodule_search_locations=list(mb.__path__))
    m = importlib.util.module_from_spec(spec)
    import sys

    sys.modules["moe_binding_fresh"] = m
    try:
        spec.loader.exec_module(m)
    finally:
        for k in [k for k in sys.modules if k.split(".")[0] == "moe_binding_fresh"]:
            del sys.modules[k]
    return m._buf


@pytest.mark.parametrize("args", [
    (T, "x", 16, None, -1), (T, "x", 16, F32, -1), (T, "x", 0, I32 + F32, -1), (None, "x", 5, F32, 0), (4096, "x", 5, F32, 0),
    (torch.empty(0), "x", 0, F32, -1), (T, "x", 16, F32, 0), (T, "x", 16, F32, 3), (T.t(), "x", 16, F32, -1),
    (T[:, :2], "x", 1, None, -1), (T[1:], "x", 12, F32, -1), (T, "x", 17, F32, -1), (T, "x", 16, I32, -1),
    (T, "name", 16, (torch.uint8, torch.bfloat16), -1), (T, "x", 1 << 40, None, -1),
    (torch.nn.Parameter(T), "x", 16, F32, -1), (T.requires_grad_(False), "x", 16, F32, -1),
])
def test_same_as_in_python(args):
    assert _outcome(_marshal.buf, args) == _outcome(_python_buf(), args)


def test_not_a_tensor():
    for bad in ("s", 1.5, [T]):
        with pytest.raises(TypeError):
            _marshal.buf(bad, "x", 1, None, 0)
    with pytest.raises(TypeError):
        _marshal.buf(T, "x", 1, None)
    with pytest.raises(TypeError):
        _marshal.buf(T, "x", "1", None, -1)
