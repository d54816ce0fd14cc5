"""The MXFP4 products at the ends of their stated ranges: tokens' codes of 2^31 bytes behind one
buffer descriptor, and rows, codes and outputs behind 2^32 elements."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
from tests import _mx_plan as mp  # noqa: E402
from tests import _ref_many as rm  # noqa: E402
from tests import test_gpu_mx as gm  # noqa: E402
from tests import test_gpu_mx_group as gg  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def _codes(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(115, 122, (M, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return q, s


def _values(q, s, rows):
    rows = torch.as_tensor(rows, device="cuda", dtype=torch.long)
    return rm.mx_values(rm.mx_unpack(to_np(q[rows])), to_np(s[rows]))


@pytest.mark.parametrize("E,I,form", [(1, 128, "tile256"), (64, 512, "tile128"), (256, 128, "tile64")])  # noqa: E741
def test_gate_up_of_the_widest_tokens(E, I, form):  # noqa: E741
    """T d / 2 = 2^31 bytes of codes: lane offsets up to the last below 2^31."""
    T, d, count = 262144, 16384, 330
    assert mp.group_form(T, E, 1, 1, 2 * I) == form and T * d // 2 == 1 << 31
    xq, xs = _codes(T, d, 1)
    w13, wv = gg._expert_weights(1, 2 * I, d, mb.MOE_W13, d, I, 2)
    tokens = np.random.default_rng(3).integers(0, T, count)
    tokens[[0, 5, 200, 329]] = T - 1, 0, T - 2, T - 1
    rows = np.full(T, -1, np.int32)
    rows[:count] = tokens
    offsets = np.array([0, count], np.int32)
    h = torch.full((T, I), 77.0, dtype=torch.bfloat16, device="cuda")
    mb.moe_mx_gate_up(gg._group(T, E, 1, 1, d, I, mb.MOE_BF16), xq, xs, gg._cuda(offsets), gg._cuda(rows), w13, h)
    torch.cuda.synchronize()
    gu, mag = rm.product(_values(xq, xs, tokens), wv[0])
    tol = rm.product_tol(mag, d)
    ref = rm.swiglu(gu[:, :I], gu[:, I:])
    t = rm.swiglu_tol(gu[:, :I], gu[:, I:], tol[:, :I], tol[:, I:])
    got = h[:count].double().cpu().numpy()
    assert (np.abs(got - ref) <= t + (np.abs(ref) + t) * 2.0**-8).all()
    assert bool((h[count:] == 77).all())


@pytest.mark.parametrize("h_type", [mb.MOE_BF16, mb.MOE_MXFP4])
def test_sorted_rows_behind_2_to_32_elements(h_type):
    """gate_up's and down's results of 2^21 sorted rows."""
    T, E, k, n, d, I = 262144, 32, 8, 32, 128, 4096  # noqa: E741
    R = T * k
    r = np.random.default_rng(5)
    counts = r.multinomial(R - 1000, np.ones(n) / n)
    counts[-1] += 1000
    offsets, rows = gg._counts_to_rows(counts, T, k, 6)
    look = np.concatenate([np.arange(40), [R // 2, R // 2 + 1], np.arange(R - 300, R)])
    expert = np.searchsorted(offsets, look, side="right") - 1
    xq, xs = _codes(T, d, 7)
    w13, wv = gg._expert_weights(n, 2 * I, d, mb.MOE_W13, d, I, 8)
    mx = h_type == mb.MOE_MXFP4
    h = torch.zeros((R, I // 2) if mx else (R, I), dtype=torch.uint8 if mx else torch.bfloat16, device="cuda")
    hs = torch.zeros((R, I // 32), dtype=torch.uint8, device="cuda") if mx else None
    mb.moe_mx_gate_up(gg._group(T, E, k, n, d, I, h_type), xq, xs, gg._cuda(offsets), gg._cuda(rows), w13, h, hs)
    torch.cuda.synchronize()
    for e in np.unique(expert):
        at = look[expert == e]
        gu, mag = rm.product(_values(xq, xs, rows[at]), wv[e])
        tol = rm.product_tol(mag, d)
        ref = rm.swiglu(gu[:, :I], gu[:, I:])
        t = rm.swiglu_tol(gu[:, :I], gu[:, I:], tol[:, :I], tol[:, I:])
        here = torch.as_tensor(at, device="cuda")
        if mx:
            gg._check_h_mx(rm.mx_unpack(to_np(h[here])), to_np(hs[here]), ref, t)
        else:
            got = h[here].double().cpu().numpy()
            assert (np.abs(got - ref) <= t + (np.abs(ref) + t) * 2.0**-8).all()
    if not mx:
        return
    # down on narrow rows, 2^33 outputs
    del h, hs
    d, I = 4096, 128  # noqa: E741
    hq, hs = _codes(R, I, 9)
    w2, wv = gg._expert_weights(n, d, I, mb.MOE_W2, d, I, 10)
    y = torch.zeros((R, d), dtype=torch.bfloat16, device="cuda")
    mb.moe_mx_down(gg._group(T, E, k, n, d, I), hq, hs, gg._cuda(offsets), w2, y)
    torch.cuda.synchronize()
    for e in np.unique(expert):
        at = look[expert == e]
        ref, mag = rm.product(_values(hq, hs, at), wv[e])
        got = y[torch.as_tensor(at, device="cuda")].double().cpu().numpy()
        assert (np.abs(got - ref) <= rm.product_tol(mag, I) + 2.0**-8 * 1.01 * np.abs(ref)).all()


@pytest.mark.parametrize("M,N,K,out", [(262144, 32768, 128, "bf16"), (262144, 20000, 200, "fp32"), (262144, 64, 32768, "fp32")])
def test_product_behind_2_to_32_elements(M, N, K, out):
    """Outputs, and rows whose codes take 2^32 bytes."""
    dims = mb.mx_dims_from(dict(M=M, N=N, K=K, out_type=gm.KIND[out]))
    Kp = rm.padded(K)
    xq, xs = _codes(M, Kp, 11)
    q, s, w = gm._weight(N, K, 12)
    packed = torch.empty(mb.moe_packed_mx_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_mx(dims, gg._cuda(q), gg._cuda(s), packed)
    ws = torch.zeros(mb.moe_mx_gemm_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    got = torch.zeros((M, N), dtype=gm.TT[out], device="cuda")
    mb.moe_mx_gemm(dims, xq, xs, packed, got, ws)
    torch.cuda.synchronize()
    look = np.concatenate([np.arange(3), [M // 2 - 1, M // 2], np.arange(M - 10, M)])
    ref, mag = rm.product(_values(xq, xs, look)[:, :K], w)
    here = got[torch.as_tensor(look, device="cuda")].double().cpu().numpy()
    assert (np.abs(here - ref) <= rm.product_tol(mag, K) + rm.half_step(out) * np.abs(ref) * 1.0001).all()
