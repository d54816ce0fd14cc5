"""The experts' kernel rule as tests/_mx_plan.py restates it, against the library's."""

import ctypes

import pytest

import moe_decode_layer_router_amd as mb
from tests import _mx_plan as mp
from tests import test_gpu_mx_group as gg

FORMS = ["few", "tile64", "tile128", "tile256"]


def _form(T, E, k, n, d, I, N):  # noqa: E741
    f = mb.lib().moeblk_mx_group_form
    f.argtypes, f.restype = [ctypes.POINTER(mb.MoeMxGroupDims), ctypes.c_int], ctypes.c_int
    return f(ctypes.byref(mb.mx_group_dims_from(dict(T=T, E=E, topk=k, n_local=n, d=d, I=I))), N)


@pytest.mark.parametrize("E,k,n", [(1, 1, 1), (8, 2, 1), (8, 8, 8), (64, 1, 3), (256, 8, 32), (256, 8, 1), (256, 1, 7), (33, 5, 31)])
def test_the_librarys_rule(E, k, n):
    seen = set()
    for T in (1, 2, 7, 16, 17, 33, 64, 100, 128, 383, 384, 385, 512, 1000, 4096, 8192, 12345, 65536, 262144):
        for N in (128, 256, 384, 512, 1024, 1920, 4096, 8192, 16384):
            got = _form(T, E, k, n, 128, 128, N)
            assert FORMS[got] == mp.group_form(T, E, k, n, N), (T, N)
            seen.add(got)
    assert len(seen) >= 3


def test_the_gpu_tests_reach_every_kernel():
    for product in ("gate_up", "down"):
        N = lambda d, I: 2 * I if product == "gate_up" else d  # noqa: E731, E741
        got = {_form(T, E, k, n, d, I, N(d, I)) for T, E, k, n, d, I, _ in gg.CASES + gg.LARGE}  # noqa: E741
        assert got == set(range(4)), product


def test_dims_out_of_range():
    assert _form(0, 8, 2, 4, 128, 128, 256) == -1
