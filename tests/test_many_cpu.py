"""The 64-bit references of the many-row path against independent forms, and the
refusals of its entry points (no GPU)."""

import ctypes

import numpy as np
import pytest
import torch

import moe_decode_layer_router_amd as mb
from tests import _ref_many as rm

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced (checks fail first)
MIS = FAKE + 4


# ------------------------------------------------------------------ references


def test_e2m1_table_from_its_bits():
    for c in range(8):
        m, e = c & 1, c >> 1
        assert rm.E2M1[c] == (m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


@pytest.mark.parametrize("amax,e", [(0.0, -127), (2.0**-130, -127), (6.999, 0), (7.0, 1), (6.0, 0), (3.5, 0), (3.4999, -1),
                                    (1.0, -2), (13.99, 1), (14.0, 2), (3.4e38, 126), (2.0**-126, -127)])
def test_mx_scale(amax, e):
    assert rm.mx_scale(np.array([amax]))[0] == e
    assert amax < 7 * 2.0**e and (e == -127 or amax >= 7 * 2.0 ** (e - 1))
    assert (rm.mx_scale(np.array([np.inf, np.nan])) == 128).all()


def test_mx_rounding_is_nearest_and_never_saturates():
    """Against a search over all values: no other value is nearer, ties go to the even code."""
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-7, 7, 4000), (rm.E2M1[1:] + rm.E2M1[:-1]) / 2, rm.E2M1, [6.9999]])
    for a, c in zip(v, rm.mx_codes(v)):
        d = np.abs(rm.E2M1 - abs(a))
        assert d[c & 7] == d.min() and (c >= 8) == bool(np.signbit(a))
        if (d == d.min()).sum() > 1:
            assert (c & 1) == 0


def test_mx_pack_round_trip_and_padding():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 77)) * np.exp2(rng.integers(-20, 20, (3, 77)))
    q, s = rm.mx_quant(x)
    assert q.shape == (3, 128) and s.shape == (3, 4) and not q[:, 77:].any() and not s[:, 3].any()
    assert np.array_equal(rm.mx_unpack(rm.mx_pack(q)), q)
    v = rm.mx_values(q, s)[:, :77]
    step = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)[:, :77]
    assert (np.abs(v - x) <= step).all()  # half of the widest step, 2
    x[1, 40] = np.nan
    q, s = rm.mx_quant(x)
    assert s[1, 1] == 255 and not q[1, 32:64].any() and np.isnan(rm.mx_values(q, s)[1, 32:64]).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gate_gradient_against_differences(score, renorm):
    """The formulas against central differences of the weights in 64 bits, an expert picked
    twice and a place without a pick among them."""
    rng = np.random.default_rng(5)
    T, E, k = 4, 7, 3
    l = (rng.standard_normal((T, E)) * 2).astype(np.float32).astype(np.float64)
    l[3] = -40.0 + 0.1 * rng.standard_normal(E)
    ids = np.argsort(-l, axis=1)[:, :k].astype(np.int32)
    ids[1, 2] = -1
    ids[2, 1] = ids[2, 0]
    g = rng.standard_normal((T, k))
    grad, mag = rm.gate_grad(l, ids, g, score, renorm)
    assert (np.abs(grad) <= mag + 1e-300).all()

    def loss(lv, t):
        slots = [s for s in range(k) if ids[t, s] >= 0]
        return float(np.dot([g[t, s] for s in slots], rm.pick_weights(lv[t], [ids[t, s] for s in slots], score, renorm)))

    h = 1e-5
    for t in range(T):
        for j in range(E):
            up, dn = l.copy(), l.copy()
            up[t, j] += h
            dn[t, j] -= h
            assert abs((loss(up, t) - loss(dn, t)) / (2 * h) - grad[t, j]) <= 1e-9 * max(1.0, abs(l[t, j])), (t, j)


def test_gate_reference_against_torch():
    """Ordinary rows: torch's top-k, sigmoid and softmax in float64."""
    rng = np.random.default_rng(2)
    l = (rng.standard_normal((50, 40)) * 3).astype(np.float32)
    tl = torch.from_numpy(l).double()
    for score in ("sigmoid", "softmax"):
        p = torch.sigmoid(tl) if score == "sigmoid" else torch.softmax(tl, dim=1)
        for renorm in (0, 1):
            ids, w = rm.gate(l, None, 6, score, renorm)
            top = torch.topk(tl, 6, dim=1).indices
            assert np.array_equal(ids, top.numpy())
            v = p.gather(1, top)
            v = v / v.sum(dim=1, keepdim=True) if renorm else v
            assert np.allclose(w, v.numpy(), rtol=1e-12, atol=0)


def test_gate_reference_at_masks():
    l = np.full((4, 5), -np.inf, np.float32)
    l[1, 3] = 2.0
    l[2] = -3e38  # the lowest values there are: weights keep their ratios
    l[3, 1] = np.nan
    l[3, 2] = 5.0
    ids, w = rm.gate(l, None, 3, "sigmoid", 1)
    assert ids.tolist() == [[-1, -1, -1], [3, -1, -1], [0, 1, 2], [1, 2, -1]]
    assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0] and np.allclose(w[2], 1 / 3)
    assert np.isnan(w[3, 0])


def test_sort_reference():
    ids = np.array([[3, 9], [2, 3], [-1, 3], [3, 3]], np.int32)
    counts, offsets, rows, pos = rm.sort_picks(ids, 2, 2)
    assert counts.tolist() == [1, 5] and offsets.tolist() == [0, 1, 6]
    assert rows.tolist() == [1, 0, 1, 2, 3, 3, -1, -1]
    assert pos.tolist() == [[1, -1], [0, 2], [-1, 3], [4, 5]]


# ------------------------------------------------------------------ refusals


def gdims(**kw):
    return mb.gate_dims_from(dict(dict(T=100, E=256, topk=8), **kw))


def rdims(**kw):
    return mb.rows_dims_from(dict(dict(T=100, E=256, topk=8, n_local=32, local_base=0, d=4096), **kw))


def xdims(**kw):
    return mb.mx_dims_from(dict(dict(M=8, N=1024, K=4096), **kw))


def grpdims(**kw):
    return mb.mx_group_dims_from(dict(dict(T=100, E=256, topk=8, n_local=32, d=4096, I=2048), **kw))


OK, SHAPE, UNSUP = mb.MOE_OK, mb.MOE_ERR_SHAPE, mb.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(T=1, E=1, topk=1), OK), (dict(T=1 << 22, score=1, renorm=0, bias_mode=1), OK),
    (dict(T=0), SHAPE), (dict(T=(1 << 22) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=257), SHAPE), (dict(topk=0), SHAPE),
    (dict(topk=9), SHAPE), (dict(E=4, topk=5), SHAPE), (dict(score=2), UNSUP), (dict(renorm=2), UNSUP),
    (dict(bias_mode=-1), UNSUP),
])
def test_check_gate_dims(kw, code):
    assert mb.moe_check_gate_dims(gdims(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(T=1, E=1, topk=1, n_local=1, d=1), OK), (dict(T=1 << 22, n_local=256, d=16384, tok_type=1, row_type=1), OK),
    (dict(local_base=224), OK), (dict(T=0), SHAPE), (dict(T=(1 << 22) + 1), SHAPE), (dict(E=257), SHAPE), (dict(E=0), SHAPE),
    (dict(topk=0), SHAPE), (dict(topk=9), SHAPE), (dict(n_local=0), SHAPE), (dict(n_local=257), SHAPE),
    (dict(local_base=-1), SHAPE), (dict(local_base=225), SHAPE), (dict(local_base=2**31 - 1), SHAPE),
    (dict(n_local=2**31 - 1), SHAPE), (dict(d=0), SHAPE), (dict(d=16385), SHAPE), (dict(tok_type=2), UNSUP),
    (dict(row_type=-1), UNSUP),
])
def test_check_rows_dims(kw, code):
    assert mb.moe_check_rows_dims(rdims(**kw)) == code
    assert (mb.moe_sort_workspace_bytes(rdims(**kw)) > 0) == (code == OK)


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(M=1, N=1, K=1), OK), (dict(M=262144, N=32768, K=32768, in_type=1, out_type=1), OK),
    (dict(M=0), SHAPE), (dict(M=262145), SHAPE), (dict(N=0), SHAPE), (dict(N=32769), SHAPE), (dict(K=0), SHAPE),
    (dict(K=32769), SHAPE), (dict(in_type=2), UNSUP), (dict(out_type=2), UNSUP), (dict(out_type=-1), UNSUP),
])
def test_check_mx_dims(kw, code):
    d = xdims(**kw)
    assert mb.moe_check_mx_dims(d) == code
    for size in (mb.moe_packed_mx_bytes, mb.moe_mx_gemm_workspace_bytes, mb.moe_mx_proj_workspace_bytes):
        assert (size(d) > 0) == (code == OK)


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(T=1, E=1, topk=1, n_local=1, d=128, I=128), OK),
    (dict(T=262144, n_local=32, d=16384, I=8192, h_type=0, out_type=1), OK), (dict(T=0), SHAPE), (dict(T=262145), SHAPE),
    (dict(E=257), SHAPE), (dict(topk=9), SHAPE), (dict(E=4, topk=5), SHAPE), (dict(n_local=33), SHAPE), (dict(n_local=0), SHAPE),
    (dict(E=16, n_local=17), SHAPE), (dict(d=64), SHAPE), (dict(d=16512), SHAPE), (dict(d=200), SHAPE), (dict(I=100), SHAPE),
    (dict(I=8320), SHAPE), (dict(h_type=1), UNSUP), (dict(out_type=2), UNSUP),
])
def test_check_mx_group_dims(kw, code):
    assert mb.moe_check_mx_group_dims(grpdims(**kw)) == code


def test_sizes():
    assert mb.moe_packed_mx_bytes(xdims()) == 1024 * 4096 * 17 // 32
    assert mb.moe_packed_mx_bytes(xdims(N=65, K=129)) == 2 * 2 * 4352  # padded rows and columns
    w = mb.dims_from(dict(S=1, d=4096, E=8, topk=1, n_local=8, local_base=0, I=2048, renorm=1, eps=1e-6, shared_I=0))
    assert mb.moe_packed_mxfp4_bytes(w, mb.MOE_W13) == 8 * mb._mx_bytes(4096, 4096)
    assert mb.moe_packed_mxfp4_bytes(w, mb.MOE_W2) == 8 * mb._mx_bytes(4096, 2048)


def _rejects(fn, dims, bad, ok, optional=(), tail=()):
    """NULL and misaligned pointers at every place, NULL and bad dims."""
    call = lambda d, a: getattr(mb.lib(), fn)(d, *a, *tail, None)  # noqa: E731
    assert call(None, ok) == mb.MOE_ERR_NULL
    assert call(ctypes.byref(bad), ok) in (SHAPE, UNSUP)
    for i in range(len(ok)):
        a = list(ok)
        if i not in optional:
            a[i] = None
            assert call(ctypes.byref(dims), a) == mb.MOE_ERR_NULL, (fn, i)
        a[i] = MIS
        assert call(ctypes.byref(dims), a) == mb.MOE_ERR_ALIGN, (fn, i)


def test_gate_calls_reject():
    _rejects("moe_gate", gdims(), gdims(E=0), [FAKE] * 4, optional=(1,))
    _rejects("moe_gate_backward", gdims(), gdims(T=0), [FAKE] * 5, optional=(3,))


def test_rows_calls_reject():
    d = rdims()
    need = mb.moe_sort_workspace_bytes(d)
    _rejects("moe_sort", d, rdims(T=0), [FAKE] * 6, tail=(need,))
    assert mb.lib().moe_sort(ctypes.byref(d), *[FAKE] * 6, need - 1, None) == mb.MOE_ERR_WORKSPACE
    _rejects("moe_dispatch", d, rdims(d=0), [FAKE] * 3)
    _rejects("moe_return", d, rdims(row_type=7), [FAKE] * 4, optional=(1,))
    _rejects("moe_return_backward", d, rdims(tok_type=7), [FAKE] * 6)


def test_mx_calls_reject():
    d = xdims()
    _rejects("moe_mx_quant", d, xdims(K=0), [FAKE] * 3)
    _rejects("moe_mx_dequant", d, xdims(M=0), [FAKE] * 3)
    _rejects("moe_pack_mx", d, xdims(N=0), [FAKE] * 3)
    need = mb.moe_mx_gemm_workspace_bytes(d)
    _rejects("moe_mx_gemm", d, xdims(M=0), [FAKE] * 5, tail=(need,))
    assert mb.lib().moe_mx_gemm(ctypes.byref(d), *[FAKE] * 5, need - 1, None) == mb.MOE_ERR_WORKSPACE
    need = mb.moe_mx_proj_workspace_bytes(d)
    _rejects("moe_mx_proj", d, xdims(out_type=3), [FAKE] * 4, tail=(need,))
    assert mb.lib().moe_mx_proj(ctypes.byref(d), *[FAKE] * 4, need - 1, None) == mb.MOE_ERR_WORKSPACE


def test_mx_group_calls_reject():
    _rejects("moe_mx_gate_up", grpdims(), grpdims(I=100), [FAKE] * 7)
    _rejects("moe_mx_gate_up", grpdims(h_type=mb.MOE_BF16), grpdims(d=1), [FAKE] * 6 + [None], optional=(6,))
    _rejects("moe_mx_down", grpdims(), grpdims(out_type=9), [FAKE] * 5)


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(16)
    for call in (lambda: mb._buf(t, "x", 16, None, 0), lambda: mb._buf(t, "x", 17, None, -1),
                 lambda: mb._buf(t, "x", 16, (torch.int32,), -1)):
        with pytest.raises(ValueError):
            call()
