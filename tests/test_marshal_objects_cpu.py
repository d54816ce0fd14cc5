"""What the binding's check in C leaves to the one in Python: objects that are no torch tensors
but answer what is asked of one, and sizes beyond 64 bits."""

import importlib.util
import subprocess
import sys

import pytest
import torch

import moe_decode_layer_router_amd as mb

F32 = (torch.float32,)


class Buffer:
    """A device buffer of another library's."""

    def __init__(self, device=0, n=16, dtype=torch.float32, contiguous=True):
        self.device, self.n, self.dtype, self.contiguous = device, n, dtype, contiguous

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.n

    def data_ptr(self):
        return 0x7F0000000000


def _buf():
    mb._t()  # puts the check in C in place, if it is built
    return mb._buf


def test_the_check_in_c_is_in_place():
    if importlib.util.find_spec("moe_decode_layer_router_amd._marshal") is None:
        pytest.skip("not built")
    assert type(_buf()).__name__ == "builtin_function_or_method"


def test_a_buffer_that_is_no_tensor():
    assert _buf()(Buffer(), "x", 16, F32, 0) == 0x7F0000000000
    assert mb._workspace(Buffer(dtype=torch.uint8, n=512), None, mb._t(), 0) == (0x7F0000000000, 512)


@pytest.mark.parametrize("bad", [dict(device=1), dict(n=15), dict(dtype=torch.int32), dict(contiguous=False)])
def test_such_a_buffer_is_checked(bad):
    with pytest.raises(ValueError, match="x: "):
        _buf()(Buffer(**bad), "x", 16, F32, 0)


class Shard(torch.Tensor):
    """A subclass with answers of its own."""

    def numel(self):
        return 4


def test_a_subclass_answers_for_itself():
    t = torch.zeros(16).as_subclass(Shard)
    assert _buf()(t, "x", 4, F32, -1) == t.data_ptr()
    with pytest.raises(ValueError, match="4 elements"):
        _buf()(t, "x", 16, F32, -1)


def test_other_objects_are_refused():
    for bad in ("s", 1.5, [torch.zeros(4)]):
        with pytest.raises((TypeError, AttributeError)):
            _buf()(bad, "x", 1, F32, 0)


@pytest.mark.parametrize("n", [2**63, 2**93, (2**31 - 1) ** 3])
def test_sizes_beyond_64_bits(n):
    """Dims far out of range ask for such sizes before the library refuses them."""
    with pytest.raises(ValueError, match="16 elements"):
        _buf()(torch.zeros(16), "x", n, F32, -1)


def test_without_the_check_in_python_it_refuses():
    """The extension alone, in a process of its own."""
    if importlib.util.find_spec("moe_decode_layer_router_amd._marshal") is None:
        pytest.skip("not built")
    code = """
import torch
from moe_decode_layer_router_amd._marshal import buf
class B:
    get_device = lambda self: 0
for args, error in (((B(), "x", 1, None, 0), TypeError), ((torch.zeros(4), "x", 2**70, None, -1), OverflowError)):
    try:
        buf(*args)
    except error:
        continue
    raise SystemExit(f"{args}: no {error}")
"""
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0


def test_two_first_calls():
    """Two threads may both find the binding's state not yet there: the check in C still leaves
    its rest to the one in Python, not to itself."""
    code = """
import moe_decode_layer_router_amd as mb
class B:
    get_device = lambda self: 0
    is_contiguous = lambda self: True
    numel = lambda self: 4
    data_ptr = lambda self: 64
for _ in range(2):
    mb._torch = None
    mb._t()
raise SystemExit(0 if mb._buf(B(), "x", 4, None, 0) == 64 else 1)
"""
    assert subprocess.run([sys.executable, "-c", code], capture_output=True).returncode == 0
