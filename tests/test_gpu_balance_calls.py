"""The balance calls where their kernels change form, and two of them at once.
Tolerances as in test_gpu_balance.py."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
from tests.test_gpu_balance import _case, _check  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("n_seq", [62, 63, 64, 65])
@pytest.mark.parametrize("T", [700, 9000])
def test_starts_in_lanes_and_in_memory(n_seq, T):
    """Up to 63 sequences lie in a wave's lanes, more are searched; empty ones at both
    ends, rows in front of the first and behind the last."""
    l, ids = _case(T, 72, 3, n_seq)
    cuts = np.sort(np.random.default_rng(n_seq).integers(5, T - 5, n_seq - 3)).tolist()
    _check(l, ids, [5, 5, *cuts, T - 5, T - 5], n_seq, "sigmoid")


@pytest.mark.parametrize("T,n_seq", [(224, 1), (225, 1), (240, 1), (241, 1), (16, 14), (16, 15), (16, 16), (209, 2)])
def test_one_launch_and_two(T, n_seq):
    """Both sides of the slots that the first launch's last workgroup sums."""
    l, ids = _case(T, 130, 4, n_seq)
    cuts = np.sort(np.random.default_rng(T).integers(0, T + 1, n_seq - 1)).tolist()
    _check(l, ids, [0, *cuts, T], n_seq, "softmax")


def test_two_streams_at_once():
    """Two batches with workspaces of their own, on two streams."""
    jobs = []
    for T, seed in ((3000, 1), (2500, 2)):
        l, ids = _case(T, 256, 8, seed)
        dims = mb.balance_dims_from(dict(T=T, E=256, topk=8, n_seq=1, coef=0.01))
        f32, i32 = dict(device="cuda"), dict(dtype=torch.int32, device="cuda")
        jobs.append(dict(
            dims=dims, l=torch.from_numpy(l).cuda(), ids=torch.from_numpy(ids).cuda(), counts=torch.empty((1, 256), **i32),
            probs=torch.empty((1, 256), **f32), loss=torch.empty(1, **f32), dl=torch.empty((T, 256), **f32),
            ws=torch.zeros(mb.moe_balance_workspace_bytes(dims), dtype=torch.uint8, device="cuda")))

    def step(j, st=None):
        mb.moe_balance_loss(j["dims"], j["l"], j["ids"], None, j["counts"], j["probs"], j["loss"], j["ws"], stream=st)
        mb.moe_balance_backward(j["dims"], j["l"], j["counts"], None, None, j["dl"], stream=st)

    out = ("counts", "probs", "loss", "dl")
    refs = []
    for j in jobs:
        step(j)
        refs.append([j[k].clone() for k in out])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        for st, j in zip(streams, jobs):
            step(j, st)
    torch.cuda.synchronize()
    for j, ref in zip(jobs, refs):
        assert all(torch.equal(j[k], r) for k, r in zip(out, ref))
