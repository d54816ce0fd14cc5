"""GPU parity of moe_sort, moe_dispatch, moe_return and moe_return_backward against the
64-bit references of tests/_ref_many.py."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
from tests import _ref_many as rm  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402

KIND = {"bf16": mb.MOE_BF16, "fp32": mb.MOE_FP32}
TT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ids(T, E, k, seed, distinct=True):
    r = np.random.default_rng([seed, T, E, k])
    if distinct:
        ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    else:
        ids = r.integers(0, E, (T, k)).astype(np.int32)
    ids[r.random((T, k)) < 0.03] = -1
    if T > 10:
        ids[T // 2] = -1
    return np.ascontiguousarray(ids)


def _dims(T, E, k, n, base, d=1, tok="bf16", row="bf16"):
    return mb.rows_dims_from(dict(T=T, E=E, topk=k, n_local=n, local_base=base, d=d, tok_type=KIND[tok], row_type=KIND[row]))


def _sort(ids, E, n, base, ws=None):
    T, k = ids.shape
    d = _dims(T, E, k, n, base)
    i32 = dict(dtype=torch.int32, device="cuda")
    sizes = (n, n + 1, T * k, T * k)
    out = [torch.full((s + 5,), 77, **i32) for s in sizes]
    if ws is None:  # no initial contents are needed
        ws = torch.full((mb.moe_sort_workspace_bytes(d),), 0xA5, dtype=torch.uint8, device="cuda")
    mb.moe_sort(d, torch.from_numpy(ids).cuda(), *out, ws)
    torch.cuda.synchronize()
    out = [to_np(o) for o in out]
    assert all((o[s:] == 77).all() for o, s in zip(out, sizes)), "wrote behind its outputs"
    counts, offsets, rows, pos = (o[:s] for o, s in zip(out, sizes))
    return counts, offsets, rows, pos.reshape(T, k)


def _check_sort(ids, E, n, base):
    for a, b in zip(_sort(ids, E, n, base), rm.sort_picks(ids, base, n)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("T,E,k,n,base", [
    (1, 1, 1, 1, 0), (1, 256, 8, 32, 64), (2, 8, 2, 8, 0), (64, 256, 8, 32, 224), (128, 256, 8, 256, 0), (255, 60, 7, 31, 3),
    (256, 256, 8, 32, 0), (257, 256, 8, 255, 1), (300, 9, 7, 3, 6), (1000, 256, 8, 32, 32), (4096, 256, 8, 256, 0),
    (8191, 64, 3, 2, 62), (65537, 256, 8, 32, 0), (70000, 16, 8, 16, 0),
])
def test_sort(T, E, k, n, base):
    _check_sort(_ids(T, E, k, 0), E, n, base)


@pytest.mark.parametrize("T", [1, 100, 3000])
def test_sort_repeated_and_foreign_ids(T):
    ids = _ids(T, 20, 5, 1, distinct=False)
    _check_sort(ids, 20, 6, 7)
    _check_sort(np.full((T, 5), 9, np.int32), 20, 6, 7)  # every pick one expert
    _check_sort(np.full((T, 5), -1, np.int32), 20, 6, 7)  # none
    ids[::2] = np.int32(2**31 - 1)
    ids[1::2] = np.int32(-2**31)
    ids[T // 2, 2] = 12
    _check_sort(ids, 20, 6, 7)


def test_sort_largest():
    """2^25 picks: against torch's stable sort."""
    T, k, E = 1 << 22, 8, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    d = _dims(T, E, k, 200, 30)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.empty(200, **i32), torch.empty(201, **i32)
    rows, pos = torch.empty(T * k, **i32), torch.empty((T, k), **i32)
    mb.moe_sort(d, ids, counts, offsets, rows, pos,
                torch.empty(mb.moe_sort_workspace_bytes(d), dtype=torch.uint8, device="cuda"))
    key = torch.where((ids >= 30) & (ids < 230), ids - 30, 200).reshape(-1)
    order = torch.sort(key, stable=True).indices
    total = int((key < 200).sum())
    assert torch.equal(counts.long(), torch.bincount(key, minlength=201)[:200])
    assert int(offsets[0]) == 0 and torch.equal(offsets[1:].long(), torch.cumsum(counts.long(), 0))
    assert torch.equal(rows[:total].long(), order[:total] // k) and bool((rows[total:] == -1).all())
    want = torch.full((T * k,), -1, device="cuda", dtype=torch.long)
    want[order[:total]] = torch.arange(total, device="cuda")
    assert torch.equal(pos.view(-1).long(), want)


def test_sort_matches_moe_bucket():
    """A decode step's picks through either call: the same buckets."""
    S, E, k, n, base = 96, 256, 8, 32, 64
    r = np.random.default_rng(4)
    ids = np.ascontiguousarray(np.argsort(r.random((S, E)), axis=1)[:, :k].astype(np.int32))
    bd = mb.dims_from(dict(S=S, d=4096, E=E, topk=k, n_local=n, local_base=base, I=2048, renorm=1, eps=1e-6, shared_I=0))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.empty(s, **i32) for s in (n, n + 1, S * k, S * k, n + 1)]
    mb.moe_bucket(bd, torch.from_numpy(ids).cuda(), *out)
    counts, offsets, rows, pos = _sort(ids, E, n, base)
    for a, b in zip((counts, offsets, rows, pos.reshape(-1)), out):
        assert np.array_equal(a, to_np(b))


# ------------------------------------------------------------------ rows


def _np64(t):
    return t.double().cpu().numpy()


def _round(v, kind):
    return _np64(torch.from_numpy(v.astype(np.float32)).to(TT[kind])) if kind == "bf16" else v


ROWS = [(1, 1, 1, 1, 1, 0), (3, 8, 6, 2, 4, 2), (40, 33, 24, 5, 8, 8), (64, 128, 16, 3, 16, 0), (20, 129, 16, 8, 3, 5),
        (50, 1000, 64, 8, 8, 40), (9, 1024, 16, 8, 16, 0), (7, 1025, 16, 8, 16, 0), (30, 4096, 256, 8, 32, 0),
        (5, 4099, 16, 4, 16, 0), (3, 16384, 8, 8, 8, 0), (600, 64, 256, 8, 128, 64)]


@pytest.mark.parametrize("tok", ["bf16", "fp32"])
@pytest.mark.parametrize("row", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,E,k,n,base", ROWS)
def test_rows(T, d, E, k, n, base, tok, row):
    ids = _ids(T, E, k, 5)
    _, offsets, _, pos = rm.sort_picks(ids, base, n)
    total, R = int(offsets[-1]), T * k
    g = torch.Generator().manual_seed(T * 7 + d)
    x = torch.randn((T, d), generator=g).to(TT[tok])
    y = torch.randn((R, d), generator=g).to(TT[row])
    y[total:] = float("nan")  # rows that no pick has
    w = torch.rand((T, k), generator=g)
    w[torch.from_numpy(pos) < 0] = float("nan")  # weights of absent picks are not looked at
    dims = _dims(T, E, k, n, base, d, tok, row)
    posd, xd, yd, wd = torch.from_numpy(pos).cuda(), x.cuda(), y.cuda(), w.cuda()
    x64, y64 = _np64(x), _np64(y)

    xs = torch.full((R, d), 77.0, dtype=TT[row], device="cuda")
    mb.moe_dispatch(dims, xd, posd, xs)
    want = np.full((R, d), 77.0)
    for s in range(k):
        on = pos[:, s] >= 0
        want[pos[on, s]] = x64[on]
    assert np.array_equal(_np64(xs), _round(want, row))

    for weights in (wd, None):
        out = torch.full((T + 1, d), 77.0, dtype=TT[tok], device="cuda")
        mb.moe_return(dims, yd, weights, posd, out)
        ref, mag = rm.weighted_sum(y64, None if weights is None else w.numpy(), pos)
        got = _np64(out)
        assert (got[T] == 77).all()
        # k fused multiply-adds, one rounding
        tol = k * rm.U24 * mag + rm.half_step(tok) * np.abs(ref) * 1.001
        assert (np.abs(got[:T] - ref) <= tol).all()
        assert (got[:T][(pos < 0).all(axis=1)] == 0).all()

    dy = torch.full((R, d), 77.0, dtype=TT[row], device="cuda")
    dw = torch.full((T + 1, k), 77.0, device="cuda")
    mb.moe_return_backward(dims, xd, yd, wd, posd, dy, dw)
    got, gw = _np64(dy), _np64(dw)
    assert (got[total:] == 77).all() and (gw[T] == 77).all()
    lanes = 16 if d <= 128 else 64 if d <= 1024 else 256
    n_add = 8 * -(-d // (8 * lanes)) + 10  # a thread's fused multiply-adds, then the tree
    for t in range(T):
        for s in range(k):
            p = pos[t, s]
            if p < 0:
                assert gw[t, s] == 0
                continue
            want = float(w[t, s]) * x64[t]
            assert (np.abs(got[p] - want) <= (rm.U24 + rm.half_step(row)) * 1.001 * np.abs(want)).all()
            terms = x64[t] * y64[p]
            assert abs(gw[t, s] - terms.sum()) <= n_add * rm.U24 * np.abs(terms).sum()


def test_return_gradient_against_differences():
    """<dout, moe_return> moves with y and topk_w as dy and dtopk_w say (fp32 throughout,
    a linear function of each: the difference over a step of 1 is exact up to rounding)."""
    T, d, E, k, n = 6, 40, 8, 3, 5
    ids = _ids(T, E, k, 6)
    _, offsets, _, pos = rm.sort_picks(ids, 2, n)
    dims = _dims(T, E, k, n, 2, d, "fp32", "fp32")
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn((T * k, d), generator=g, device="cuda")
    w = torch.rand((T, k), generator=g, device="cuda")
    dout = torch.randn((T, d), generator=g, device="cuda")
    posd = torch.from_numpy(pos).cuda()
    out = torch.empty((T, d), device="cuda")

    def f():
        mb.moe_return(dims, y, w, posd, out)
        return float((out.double() * dout.double()).sum())

    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    mb.moe_return_backward(dims, dout, y, w, posd, dy, dw)
    base = f()
    tol = 64 * d * T * rm.U24
    for t in range(T):
        for s in range(k):
            w[t, s] += 1
            assert abs(f() - base - float(dw[t, s])) <= tol
            w[t, s] -= 1
    for r in range(int(offsets[-1])):
        for c in (0, 17, d - 1):
            y[r, c] += 1
            assert abs(f() - base - float(dy[r, c])) <= tol
            y[r, c] -= 1


def test_rows_positions_outside_are_none():
    """A position behind the sorted rows is no pick: nothing is read or written there."""
    T, k, d = 4, 3, 32
    dims = _dims(T, 8, k, 8, 0, d, "fp32", "fp32")
    pos = torch.tensor([[0, 12, 1], [-5, 2, 10**9], [3, 4, 5], [-1, -1, 2**31 - 1]], dtype=torch.int32, device="cuda")
    x = torch.randn((T, d), device="cuda")
    big = torch.full((T * k + 64, d), 77.0, device="cuda")
    mb.moe_dispatch(dims, x, pos, big)
    assert bool((big[6:] == 77).all()) and torch.equal(big[0], x[0]) and torch.equal(big[2], x[1])
    out = torch.empty((T, d), device="cuda")
    mb.moe_return(dims, big, None, pos, out)
    assert torch.equal(out[0], 2 * x[0]) and torch.equal(out[1], x[1]) and not bool(out[3].any())


def test_rows_behind_2_to_32_elements():
    T, k, d = 40000, 8, 16384
    R = T * k
    dims = _dims(T, 8, k, 8, 0, d, "bf16", "bf16")
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    pos = torch.arange(R, device="cuda", dtype=torch.int32).view(T, k).flip(0).contiguous()
    xs = torch.empty((R, d), dtype=torch.bfloat16, device="cuda")
    mb.moe_dispatch(dims, x, pos, xs)
    for t in (0, 1, T // 2, T - 1):
        for s in (0, k - 1):
            assert torch.equal(xs[int(pos[t, s])], x[t])
    w = torch.full((T, k), 0.125, device="cuda")
    out = torch.empty_like(x)
    mb.moe_return(dims, xs, w, pos, out)
    assert torch.equal(out, x)
