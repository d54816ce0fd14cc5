"""The 64-bit references of the FP8 products and the balance loss against
independent forms, and the refusals of their entry points (no GPU)."""

import ctypes

import numpy as np
import pytest
import torch

import moe_decode_layer_router_amd as mb
from synth import CONFIGS
from tests import _ref_fp8 as rf

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced (checks fail first)
MIS = FAKE + 4


# ------------------------------------------------------------------ references


def test_e4m3_table_and_encoding_match_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, rf.TABLE, equal_nan=True)
    rng = np.random.default_rng(0)
    v = rng.standard_normal(20000) * np.exp2(rng.uniform(-14, 8, 20000))
    v = np.clip(np.concatenate([v, rf.TABLE[:127], -rf.TABLE[:127], rf._MID, -rf._MID]), -448, 448)
    v = v.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(rf.e4m3_encode(v), want)


@pytest.mark.parametrize("amax,e", [(0.0, -126), (448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (1.0, -8),
                                    (2.0**-130, -126), (3.3e38, 120)])
def test_block_scale(amax, e):
    assert rf.block_scale(np.array([amax]))[0] == 2.0**e
    assert np.isnan(rf.block_scale(np.array([np.inf, np.nan]))).all()


def test_quant_pads_and_marks_blocks_that_are_not_finite():
    x = np.ones((2, 130))
    x[1, 129] = np.nan
    q, s = rf.quant(x)
    assert q.shape == (2, 256) and s.shape == (2, 2)
    assert not q[0, 130:].any()
    assert np.isnan(s[1, 1]) and np.isnan(rf.TABLE[q[1, 128:]]).all() and np.isfinite(s[0]).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_balance_gradient_against_differences(score):
    """The formula's gradient against central differences of the loss in 64
    bits: truncation ~ h^2, rounding ~ 2^-52 L / h."""
    rng = np.random.default_rng(3)
    T, E, k = 9, 7, 2
    l = rng.standard_normal((T, E)) * 2
    ids = np.argsort(-l, axis=1)[:, :k].astype(np.int32)
    starts = [1, 4, 4, 8]
    h = 1e-5
    args = (ids, starts, 3, score, 0.7)
    grad = rf.balance(l, *args)[3]
    assert np.isnan(grad[0]).all() and np.isnan(grad[8]).all()
    for t in range(1, 8):
        for j in range(E):
            up, dn = l.copy(), l.copy()
            up[t, j] += h
            dn[t, j] -= h
            d = (rf.balance(up, *args)[2] - rf.balance(dn, *args)[2]) / (2 * h)
            assert abs(d - grad[t, j]) <= 1e-9, (t, j)


def test_balance_of_even_routing_is_coef():
    """Every expert picked equally often under uniform scores: sum_e f P = 1."""
    E, k = 8, 2
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(4)], np.int32)
    c, p, loss, g = rf.balance(np.zeros((4, E)), ids, [0, 4], 1, "softmax", 0.3)
    assert np.all(c == 1) and np.allclose(p, 1 / E) and abs(loss - 0.3) < 1e-15 and np.abs(g).max() < 1e-17


# ------------------------------------------------------------------ refusals


def fdims(**kw):
    return mb.fp8_dims_from(dict(dict(M=8, N=1024, K=4096), **kw))


def bdims(**kw):
    return mb.balance_dims_from(dict(dict(T=100, E=256, topk=8, n_seq=1), **kw))


def edims(**kw):
    return mb.dims_from(dict(CONFIGS["s8_uniform"].dims(), **kw))


@pytest.mark.parametrize("kw,code", [
    (dict(), mb.MOE_OK),
    (dict(M=1, N=1, K=1), mb.MOE_OK),
    (dict(M=262144, N=32768, K=32768, in_type=1, out_type=1), mb.MOE_OK),
    (dict(M=0), mb.MOE_ERR_SHAPE),
    (dict(M=262145), mb.MOE_ERR_SHAPE),
    (dict(N=0), mb.MOE_ERR_SHAPE),
    (dict(N=32769), mb.MOE_ERR_SHAPE),
    (dict(K=0), mb.MOE_ERR_SHAPE),
    (dict(K=-5), mb.MOE_ERR_SHAPE),
    (dict(K=32769), mb.MOE_ERR_SHAPE),
    (dict(in_type=2), mb.MOE_ERR_UNSUPPORTED),
    (dict(out_type=-1), mb.MOE_ERR_UNSUPPORTED),
])
def test_check_fp8_dims(kw, code):
    assert mb.moe_check_fp8_dims(fdims(**kw)) == code
    if code != mb.MOE_OK:
        d = fdims(**kw)
        assert mb.moe_packed_fp8_bytes(d) == 0 and mb.moe_fp8_gemm_workspace_bytes(d) == 0
        assert mb.moe_fp8_proj_workspace_bytes(d) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(), mb.MOE_OK),
    (dict(T=1, E=1, topk=1), mb.MOE_OK),
    (dict(T=1 << 22, n_seq=4096, score=1), mb.MOE_OK),
    (dict(T=0), mb.MOE_ERR_SHAPE),
    (dict(T=(1 << 22) + 1), mb.MOE_ERR_SHAPE),
    (dict(E=0), mb.MOE_ERR_SHAPE),
    (dict(E=257), mb.MOE_ERR_SHAPE),
    (dict(topk=9), mb.MOE_ERR_SHAPE),
    (dict(E=4, topk=5), mb.MOE_ERR_SHAPE),
    (dict(n_seq=0), mb.MOE_ERR_SHAPE),
    (dict(n_seq=4097), mb.MOE_ERR_SHAPE),
    (dict(score=2), mb.MOE_ERR_UNSUPPORTED),
    (dict(coef=float("nan")), mb.MOE_ERR_UNSUPPORTED),
    (dict(coef=float("inf")), mb.MOE_ERR_UNSUPPORTED),
])
def test_check_balance_dims(kw, code):
    assert mb.moe_check_balance_dims(bdims(**kw)) == code
    assert (mb.moe_balance_workspace_bytes(bdims(**kw)) > 0) == (code == mb.MOE_OK)


def test_sizes():
    assert mb.moe_packed_fp8_bytes(fdims()) == 1024 * 4096 + 8 * 32 * 4
    assert mb.moe_packed_fp8_bytes(fdims(N=65, K=129)) == 128 * 256 + 16  # padded rows and columns, 1 x 2 scales
    d = edims()
    assert mb.moe_packed_fp8_expert_bytes(d, mb.MOE_W13) == 32 * (4096 * 4096 + 32 * 32 * 4)
    assert mb.moe_packed_fp8_expert_bytes(d, mb.MOE_W2) == 32 * (4096 * 2048 + 32 * 16 * 4)
    assert mb.moe_packed_fp8_expert_bytes(d, mb.MOE_WS13) == 0  # no shared expert
    assert mb.moe_packed_fp8_expert_bytes(d, 4) == mb.moe_packed_fp8_expert_bytes(d, -1) == 0
    d4 = mb.dims_from(CONFIGS["s128_shared"])
    assert mb.moe_packed_fp8_expert_bytes(d4, mb.MOE_WS2) == 7168 * 2048 + 56 * 16 * 4
    assert mb.moe_fp8_ffn_workspace_bytes(d4) % 16 == 0
    assert mb.moe_fp8_ffn_workspace_bytes(edims(S=0)) == 0


def _rejects(fn, dims, bad, ok, optional=(), tail=()):
    """NULL and misaligned pointers at every place, NULL and bad dims."""
    call = lambda d, a: getattr(mb.lib(), fn)(d, *a, *tail, None)  # noqa: E731
    assert call(None, ok) == mb.MOE_ERR_NULL
    assert call(ctypes.byref(bad), ok) in (mb.MOE_ERR_SHAPE, mb.MOE_ERR_UNSUPPORTED)
    for i in range(len(ok)):
        a = list(ok)
        if i not in optional:
            a[i] = None
            assert call(ctypes.byref(dims), a) == mb.MOE_ERR_NULL, (fn, i)
        a[i] = MIS
        assert call(ctypes.byref(dims), a) == mb.MOE_ERR_ALIGN, (fn, i)


def test_fp8_calls_reject():
    d = fdims()
    _rejects("moe_fp8_quant", d, fdims(K=0), [FAKE] * 3)
    _rejects("moe_pack_fp8", d, fdims(N=0), [FAKE] * 3)
    need = mb.moe_fp8_gemm_workspace_bytes(d)
    _rejects("moe_fp8_gemm", d, fdims(M=0), [FAKE] * 5, tail=(need,))
    assert mb.lib().moe_fp8_gemm(ctypes.byref(d), *[FAKE] * 5, need - 1, None) == mb.MOE_ERR_WORKSPACE
    need = mb.moe_fp8_proj_workspace_bytes(d)
    _rejects("moe_fp8_proj", d, fdims(out_type=3), [FAKE] * 4, tail=(need,))
    assert mb.lib().moe_fp8_proj(ctypes.byref(d), *[FAKE] * 4, need - 1, None) == mb.MOE_ERR_WORKSPACE


def test_fp8_expert_calls_reject():
    d = edims()
    L = mb.lib()
    for which in (-1, 4, mb.MOE_WS13, mb.MOE_WS2):  # no shared expert in these dims
        assert L.moe_pack_fp8_expert(ctypes.byref(d), which, FAKE, FAKE, FAKE, None) == mb.MOE_ERR_UNSUPPORTED
    assert L.moe_pack_fp8_expert(None, 0, FAKE, FAKE, FAKE, None) == mb.MOE_ERR_NULL
    assert L.moe_pack_fp8_expert(ctypes.byref(d), 0, FAKE, None, FAKE, None) == mb.MOE_ERR_NULL
    assert L.moe_pack_fp8_expert(ctypes.byref(d), 1, FAKE, MIS, FAKE, None) == mb.MOE_ERR_ALIGN
    need = mb.moe_fp8_ffn_workspace_bytes(d)
    ok = [FAKE] * 7 + [None, None, FAKE, FAKE]
    _rejects("moe_fp8_expert_ffn", d, edims(I=100), ok, optional=(7, 8), tail=(need,))
    assert L.moe_fp8_expert_ffn(ctypes.byref(d), *ok, need - 1, None) == mb.MOE_ERR_WORKSPACE
    d4 = mb.dims_from(CONFIGS["s128_shared"])  # a shared expert needs its weights
    assert L.moe_fp8_expert_ffn(ctypes.byref(d4), *ok, mb.moe_fp8_ffn_workspace_bytes(d4), None) == mb.MOE_ERR_NULL


def test_balance_calls_reject():
    d = bdims()
    need = mb.moe_balance_workspace_bytes(d)
    L = mb.lib()
    _rejects("moe_expert_counts", d, bdims(E=0), [FAKE, None, FAKE, FAKE], optional=(1,), tail=(need,))
    _rejects("moe_balance_loss", d, bdims(T=0), [FAKE, FAKE, None] + [FAKE] * 4, optional=(2,), tail=(need,))
    assert L.moe_balance_loss(ctypes.byref(d), *[FAKE] * 7, need - 1, None) == mb.MOE_ERR_WORKSPACE
    _rejects("moe_balance_backward", d, bdims(score=9), [FAKE, FAKE, None, None, FAKE], optional=(2, 3))
    two = bdims(n_seq=2)  # several sequences need their starts
    need = mb.moe_balance_workspace_bytes(two)
    assert L.moe_expert_counts(ctypes.byref(two), FAKE, None, FAKE, FAKE, need, None) == mb.MOE_ERR_NULL
    assert L.moe_balance_backward(ctypes.byref(two), FAKE, FAKE, None, None, FAKE, None) == mb.MOE_ERR_NULL
