"""GPU parity of the per-expert counts, the balance loss and its gradient
against the 64-bit reference of tests/_ref_fp8.py.

Tolerances (u = 2^-24): a row's p is a quotient of an fp32 exponential (2 ulp of
error, and its argument's rounding: 2 u |l|) and a sum of E of them (at most
10 additions deep, 2 u |l| of their arguments): relative error at most
(24 + 4 |l|_max) u =: r. probs adds at most 18 additions in fp32, then fp64:
(r + 20 u) P. The loss takes that relative error of its non-negative terms
and one rounding. The gradient slope_j (a_j - m): each factor to r + 4 u, m a
sum of E products (10 additions): |d| <= (2 r + 16 u) slope_j (|a_j| + m)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
from tests import _ref_fp8 as rf  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402

SCORES = {"sigmoid": mb.MOE_SCORE_SIGMOID, "softmax": mb.MOE_SCORE_SOFTMAX}
U = 2.0**-24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _run(l, ids, starts, n_seq, score, coef=0.01, dloss=None, ws=None):
    T, E = l.shape
    k = ids.shape[1]
    dims = mb.balance_dims_from(dict(T=T, E=E, topk=k, n_seq=n_seq, score=SCORES[score], coef=coef))
    if ws is None:
        ws = torch.zeros(mb.moe_balance_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    lg = torch.from_numpy(np.ascontiguousarray(l, np.float32)).cuda()
    ig = torch.from_numpy(np.ascontiguousarray(ids, np.int32)).cuda()
    sg = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    dg = None if dloss is None else torch.tensor([dloss], dtype=torch.float32, device="cuda")
    counts = torch.full((n_seq + 1, E), -9, dtype=torch.int32, device="cuda")
    probs = torch.full((n_seq + 1, E), float("nan"), device="cuda")
    loss = torch.full((4,), float("nan"), device="cuda")
    dl = torch.full((T + 1, E), 123.0, device="cuda")
    mb.moe_balance_loss(dims, lg, ig, sg, counts, probs, loss, ws)
    mb.moe_balance_backward(dims, lg, counts, sg, dg, dl)
    only = torch.full((n_seq + 1, E), -9, dtype=torch.int32, device="cuda")
    mb.moe_expert_counts(dims, ig, sg, only, ws)
    torch.cuda.synchronize()
    assert bool((counts[n_seq] == -9).all()) and bool(torch.isnan(probs[n_seq]).all())
    assert bool((dl[T] == 123.0).all()) and bool(torch.isnan(loss[1:]).all()), "wrote behind an output"
    assert torch.equal(only, counts)
    return to_np(counts)[:n_seq], to_np(probs)[:n_seq], float(loss[0]), to_np(dl)[:T]


def _check(l, ids, starts, n_seq, score, coef=0.01, dloss=None, ws=None):
    l = np.ascontiguousarray(l, np.float32)
    got = _run(l, ids, starts, n_seq, score, coef, dloss, ws)
    st = [0, l.shape[0]] if starts is None else starts
    g = 1.0 if dloss is None else dloss
    c, p, L, grad = rf.balance(l.astype(np.float64), ids, st, n_seq, score, coef, g)
    assert np.array_equal(got[0], c)
    fin = l[np.isfinite(l)]
    r = (24 + 4 * (min(float(np.abs(fin).max()), 104.0) if fin.size else 0.0)) * U
    tiny = 2.0**-126  # results below the smallest normal number
    assert np.all(np.abs(got[1] - p) <= (r + 20 * U) * p + tiny)
    assert abs(got[2] - L) <= (r + 21 * U) * abs(L) + tiny
    E, k = l.shape[1], ids.shape[1]
    inside = np.zeros(l.shape[0], bool)
    for b in range(n_seq):
        a, z = st[b], st[b + 1]
        if z <= a:
            continue
        inside[a:z] = True
        w = abs(g * coef) / n_seq * E / (k * (z - a) ** 2) * c[b]
        pr, f = rf.balance_scores(l[a:z].astype(np.float64), score)
        tol = (2 * r + 16 * U) * pr * f * (w[None, :] + (pr @ w)[:, None]) + tiny
        assert np.all(np.abs(got[3][a:z] - grad[a:z]) <= tol), (b, float((np.abs(got[3][a:z] - grad[a:z]) / tol).max()))
    assert np.all(got[3][~inside] == 123.0), "gradient rows outside the sequences were written"
    return got


def _case(T, E, k, seed, spread=2.0):
    r = np.random.default_rng([seed, T, E])
    l = (r.standard_normal((T, E)) * spread + r.standard_normal((1, E))).astype(np.float32)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    return l, ids


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 5, 2), (64, 256, 8), (65, 255, 8), (128, 256, 8),
                                   (100, 60, 6), (200, 64, 1), (1000, 65, 4), (4099, 128, 2)])
def test_one_sequence(T, E, k, score):
    l, ids = _case(T, E, k, 0)
    _check(l, ids, None, 1, score)
    _check(l, ids, [0, T], 1, score, coef=-2.5, dloss=0.3)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("starts", [
    [0, 300], [0, 0, 300], [5, 100, 290], [0, 64, 128, 192], [0, 63, 64, 65, 129, 300], [7, 7, 7, 7],
    [0, 1, 2, 3, 3, 3, 4, 250], [299, 300], [300, 300, 300], [0, 300, 300],
])
def test_sequences(starts, score):
    l, ids = _case(300, 96, 3, 1)
    _check(l, ids, starts, len(starts) - 1, score)


def test_many_sequences():
    T = 5000
    l, ids = _case(T, 40, 2, 2)
    cuts = np.sort(np.random.default_rng(0).integers(0, T + 1, 1499)).tolist()
    _check(l, ids, [0, *cuts, T], 1500, "sigmoid")


@pytest.mark.parametrize("T,E,k,n_seq", [(20000, 64, 4, 1), (9000, 255, 8, 16), (9000, 250, 8, 17), (9000, 33, 2, 700)])
def test_sums_of_many_slots(T, E, k, n_seq):
    """Sequences of many slots, and more sequences than workgroups that sum them."""
    l, ids = _case(T, E, k, 8)
    cuts = np.sort(np.random.default_rng(n_seq).integers(0, T + 1, n_seq - 1)).tolist()
    _check(l, ids, [0, *cuts, T], n_seq, "softmax")


def test_starts_outside_the_rows_are_clamped():
    l, ids = _case(100, 16, 2, 3)
    a = _run(l, ids, [-5, 40, 500], 2, "softmax")
    b = _run(l, ids, [0, 40, 100], 2, "softmax")
    for x, y in zip(a, b):
        assert np.array_equal(x, y)


def test_ids_that_are_not_experts():
    l, ids = _case(70, 32, 4, 4)
    ids[::3, 1] = -1
    ids[1::5, 2] = 32
    ids[2::7, 3] = 2**31 - 1
    ids[4, :] = 6  # the same expert four times
    _check(l, ids, [0, 30, 70], 2, "sigmoid")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_and_extreme_logits(score):
    """Masked experts (-inf, the type's lowest value), rows with nothing left,
    logits far below zero (every sigmoid vanishes in fp32) and far above."""
    l, ids = _case(140, 48, 4, 5)
    l[:, 7] = -np.inf
    l[3] = -np.inf
    l[70:74] = -np.inf
    l[5, 1:] = -np.inf
    l[8] -= 300.0
    l[9] = -1e4 + np.arange(48)
    l[10] = 90.0
    l[11, ::2] = np.finfo(np.float32).min
    l[12] = np.finfo(np.float32).min
    l[13] = 0.0
    l[14, 0] = 100.0
    _check(l, ids, [0, 20, 70, 74, 140], 4, score)


def test_nan_stays_in_its_sequence():
    l, ids = _case(128, 16, 2, 6)
    l[100, 3] = np.nan
    c, p, L, d = _run(l, ids, [0, 50, 128], 2, "softmax")
    assert np.isfinite(p[0]).all() and np.isnan(p[1]).all() and np.isnan(L)
    bad = np.isnan(d).any(axis=1)
    assert bad[100] and bad.sum() == 1


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_nan_among_masked_experts(score):
    """One NaN in a row whose other logits are all -inf: the row's p and gradient
    are NaN, the loss with them; other rows are as without it."""
    l, ids = _case(200, 96, 2, 7)
    l[150] = -np.inf
    want = _check(l, ids, [0, 100, 200], 2, score)
    l[150, 5] = np.nan
    c, p, L, d = _run(l, ids, [0, 100, 200], 2, score)
    assert np.array_equal(c, want[0]) and np.array_equal(p[0], want[1][0])
    assert np.isnan(p[1]).all() and np.isnan(L) and np.isnan(d[150]).all()
    rest = np.arange(200) != 150
    assert np.array_equal(d[rest], want[3][rest])


def test_gradient_against_differences_of_the_loss():
    """Directional central differences of the GPU's own fp32 loss: the error is
    the loss's rounding (2^-24 L, twice, over 2 h) and h^2 |d3L| / 6; the third
    derivative along a unit direction is at most 8 coef (p's are bounded by 1
    and the loss by coef E / k times them)."""
    l, ids = _case(6, 8, 2, 7, spread=1.0)
    h = 2e-2
    r = np.random.default_rng(1)
    for score in SCORES:
        base = _run(l, ids, [0, 4, 6], 2, score, coef=1.0)
        for _ in range(5):
            v = r.standard_normal(l.shape)
            v /= np.linalg.norm(v)
            up = _run(l + h * v, ids, [0, 4, 6], 2, score, coef=1.0)[2]
            dn = _run(l - h * v, ids, [0, 4, 6], 2, score, coef=1.0)[2]
            # l +- h v is rounded to fp32: 2^-24 |l| a value, through the gradient
            tol = 4 * U * abs(base[2]) / h + 8 * h * h / 6 + U * np.abs(l).max() * np.abs(base[3]).sum() / h
            assert abs((up - dn) / (2 * h) - float((base[3] * v).sum())) <= tol


def test_one_workspace_serves_other_dims_and_graphs():
    big, ids_b = _case(3000, 256, 8, 8)
    small, ids_s = _case(9, 16, 2, 8)
    dims = mb.balance_dims_from(dict(T=3000, E=256, topk=8, n_seq=3, score=0, coef=0.01))
    ws = torch.zeros(mb.moe_balance_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        _check(big, ids_b, [0, 10, 2000, 3000], 3, "sigmoid", ws=ws)
        _check(small, ids_s, None, 1, "softmax", ws=ws)
    lg, ig = torch.from_numpy(big).cuda(), torch.from_numpy(ids_b).cuda()
    sg = torch.tensor([0, 10, 2000, 3000], dtype=torch.int32, device="cuda")
    out = dict(counts=torch.empty((3, 256), dtype=torch.int32, device="cuda"), probs=torch.empty((3, 256), device="cuda"),
               loss=torch.empty(1, device="cuda"), dl=torch.empty((3000, 256), device="cuda"))

    def step():
        mb.moe_balance_loss(dims, lg, ig, sg, out["counts"], out["probs"], out["loss"], ws)
        mb.moe_balance_backward(dims, lg, out["counts"], sg, None, out["dl"])

    step()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in out.items()}
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            step()
        graphs.append(g)
    for i in range(4):
        for v in out.values():
            v.fill_(-1)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], ref[k]) for k in ref), i
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], ref[k]) for k in ref), (i, "eager")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_even_load_has_no_gradient(score):
    """Every expert picked equally often: a_j - sum a p is zero in exact
    arithmetic, and has to be zero here, not the rounding of its terms."""
    l, ids = _case(500, 8, 8, 10)  # top-8 of 8
    got = _check(l, ids, [0, 200, 500], 2, score, coef=100.0)
    assert not got[3].any()
    l, _ = _case(512, 64, 2, 11)
    ids = (np.arange(1024) % 64).reshape(512, 2).astype(np.int32)
    assert not _check(l, ids, None, 1, score)[3].any()


def test_near_even_load_keeps_its_digits():
    """One pick more on one expert: the gradient is a difference of nearly equal
    terms, still good to the bound of its own size: p f |c_j - mean| instead of p f
    |c_j| (the counts against their mean, at most 1 apart here, r and u as above)."""
    E, T = 64, 4096
    l, _ = _case(T, E, 1, 12)
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    ids[0] = 1
    got = _run(l, ids, None, 1, "softmax", coef=1.0)[3]
    c, _, _, grad = rf.balance(l.astype(np.float64), ids, [0, T], 1, "softmax", 1.0)
    w = np.abs(c[0] - T // E) * E / T**2
    p, f = rf.balance_scores(l.astype(np.float64), "softmax")
    r = (24 + 4 * float(np.abs(l).max())) * U
    tol = (2 * r + 16 * U) * p * f * (w[None, :] + (p @ w)[:, None])
    assert np.all(np.abs(got - grad) <= tol + 1e-12 * np.abs(grad) + 2.0**-50 * E / T**2)


def test_large_offsets():
    """dlogits and logits past 2^31 bytes: the last rows of 2.4e6 x 256."""
    T, E, k = 2400000, 256, 1
    dims = mb.balance_dims_from(dict(T=T, E=E, topk=k, n_seq=2, score=1, coef=1.0))
    lg = torch.zeros((T, E), device="cuda")
    ig = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    tail = 40
    l, ids = _case(tail, E, k, 9)
    lg[-tail:] = torch.from_numpy(l).cuda()
    ig[-tail:] = torch.from_numpy(ids).cuda()
    sg = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    counts = torch.empty((2, E), dtype=torch.int32, device="cuda")
    probs, loss = torch.empty((2, E), device="cuda"), torch.empty(1, device="cuda")
    dl = torch.empty((T, E), device="cuda")
    ws = torch.zeros(mb.moe_balance_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_balance_loss(dims, lg, ig, sg, counts, probs, loss, ws)
    mb.moe_balance_backward(dims, lg, counts, sg, None, dl)
    torch.cuda.synchronize()
    c, p, L, grad = rf.balance(l.astype(np.float64), ids, [0, tail], 1, "softmax", 0.5)  # half of coef: one of two
    assert np.array_equal(to_np(counts)[1], c[0]) and int(counts[0, 0]) == T - tail
    assert np.abs(to_np(probs)[1] - p[0]).max() <= 1e-5 * p.max()
    assert np.abs(to_np(probs)[0] - 1 / E).max() <= 1e-5 / E
    assert np.abs(to_np(dl[-tail:]) - grad).max() <= 1e-5 * np.abs(grad).max()


def test_binding_refuses():
    l, ids = _case(10, 16, 2, 1)
    dims = mb.balance_dims_from(dict(T=10, E=16, topk=2))
    lg, ig = torch.from_numpy(l).cuda(), torch.from_numpy(ids).cuda()
    counts = torch.empty((1, 16), dtype=torch.int32, device="cuda")
    probs, loss = torch.empty((1, 16), device="cuda"), torch.empty(1, device="cuda")
    ws = torch.zeros(mb.moe_balance_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    for a in [(lg.double(), ig), (lg.cpu(), ig), (lg[:5], ig), (lg.t(), ig), (lg, ig.long()), (lg, ig[:, :1].contiguous())]:
        with pytest.raises(ValueError):
            mb.moe_balance_loss(dims, *a, None, counts, probs, loss, ws)
    with pytest.raises(mb.MoeError) as e:
        mb.moe_balance_loss(dims, lg, ig, None, counts, probs, loss, ws[:256])
    assert e.value.code == mb.MOE_ERR_WORKSPACE
