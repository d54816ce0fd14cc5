"""moe_gate_backward works with the very weights that moe_gate gives, and what either makes of
logits that are not finite."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import _ref_many as rm  # noqa: E402
from tests import test_gpu_gate as gg  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("E", [9, 64, 100, 256])
def test_softmax_weights_bit_for_bit(E):
    """One pick of two equal largest logits: its weight is w = fl(1 / total), and with a
    gradient of one the other's dlogits is -fl(w / total). So the total can be read from
    either: some fp32 number has to give both."""
    T = 4000
    l = gg._logits(T, E, 11, spread=2.0)
    top = l.max(axis=1) + np.float32(0.25)
    l[:, 2], l[:, E - 1] = top, top
    ids, w = gg._run(l, 1, "softmax", 0)
    assert (ids == 2).all()
    w = w[:, 0].astype(np.float32)
    d = -gg._grad(l, ids, np.ones((T, 1), np.float32), "softmax", 0)[:, E - 1].astype(np.float32)
    total = (np.float32(1) / w).view(np.int32)[:, None] + np.arange(-4, 5, dtype=np.int32)
    total = total.view(np.float32)
    agree = (np.float32(1) / total == w[:, None]) & (w[:, None] / total == d[:, None])
    assert agree.any(axis=1).all(), f"{(~agree.any(axis=1)).sum()} of {T} rows"


def _not_finite(T, E):
    l = gg._logits(T, E, 12)
    l[1, 3] = np.nan
    l[2, E - 1] = -np.nan
    l[3, 0] = np.inf
    l[4, 1:4] = np.inf
    l[5] = np.inf
    l[6] = np.nan
    l[7, 2], l[7, 5] = np.nan, np.inf
    l[8] = -np.inf
    l[9, 4:] = -np.inf
    l[10, 3] = np.inf
    l[10, 6:] = -np.inf
    return l


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("E", [8, 100, 256])
def test_weights_of_logits_that_are_not_finite(E, score, renorm):
    l = _not_finite(40, E)
    with np.errstate(invalid="ignore"):
        gg._check(l, 4, score, renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("E", [8, 100, 256])
def test_gradient_of_logits_that_are_not_finite(E, score, renorm):
    """NaN where the formula has it and nowhere else; other rows keep their values."""
    T, k = 40, 4
    l = _not_finite(T, E)
    r = np.random.default_rng([13, E])
    g = r.standard_normal((T, k)).astype(np.float32)
    picked = gg._run(l, k, score, renorm)[0]
    others = r.integers(-1, E, (T, k)).astype(np.int32)
    others[3, 0], others[4, 1], others[9, 2], others[10, :2] = 0, 2, 6, (3, 7)
    others[13] = -1
    l[13, 2] = np.nan  # a row without a pick
    for ids in (picked, others):
        got = gg._grad(l, ids, g, score, renorm)
        with np.errstate(invalid="ignore", over="ignore"):
            want, mag = rm.gate_grad(l, ids, g, score, renorm)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        tol = (rm.gate_rel(l) * 2 + 20 * rm.U24) * mag + 2.0**-120
        ok = np.abs(got - want) <= tol
        assert ok[~np.isnan(want)].all()
