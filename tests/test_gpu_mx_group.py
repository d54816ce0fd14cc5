"""GPU parity of moe_mx_gate_up and moe_mx_down against the 64-bit references of
tests/_ref_many.py, and the many-row path as one: gate, sort, experts, return and their
gradients, eagerly, on streams and in a graph."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
from tests import _ref_many as rm  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _group(T, E, k, n, d, I, h_type=mb.MOE_MXFP4, out_type=mb.MOE_BF16):  # noqa: E741
    return mb.mx_group_dims_from(dict(T=T, E=E, topk=k, n_local=n, d=d, I=I, h_type=h_type, out_type=out_type))


def _expert_weights(n, N, K, which, d, I, seed):  # noqa: E741
    """Packed as the decode path packs them, and the values [n, N, K]."""
    r = np.random.default_rng([seed, n, N, K])
    code = r.integers(0, 16, (n, N, K)).astype(np.uint8)
    s = r.integers(113, 120, (n, N, K // 32)).astype(np.uint8)
    wd = mb.dims_from(dict(S=1, d=d, E=n, topk=1, n_local=n, local_base=0, I=I, renorm=1, eps=1e-6, shared_I=0))
    packed = torch.empty(mb.moe_packed_mxfp4_bytes(wd, which), dtype=torch.uint8, device="cuda")
    mb.moe_pack_mxfp4(wd, which, _cuda(rm.mx_pack(code)), _cuda(s), packed)
    return packed, rm.mx_values(code, s)


def _counts_to_rows(counts, T, k, seed):
    """offsets, rows for given counts: tokens drawn at random."""
    r = np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = np.full(T * k, -1, np.int32)
    rows[:offsets[-1]] = r.integers(0, T, offsets[-1])
    return offsets, rows


def _x(T, d, seed):
    r = np.random.default_rng([seed, T, d])
    code, s = rm.mx_quant(r.standard_normal((T, d)) * np.exp(0.5 * r.standard_normal((T, 1))))
    return code, s


def _check_h_mx(code, s, h, tol):
    """MXFP4 values of h known to within tol: each is h's nearest on the block's grid, whose
    scale is that of an amax within tol."""
    b = lambda v: v.reshape(v.shape[0], -1, 32)  # noqa: E731
    amax, slack = np.abs(b(h)).max(axis=2), b(tol).max(axis=2)
    lo, hi = rm.mx_scale(np.maximum(amax - slack, 0.0)) + 127, rm.mx_scale(amax + slack) + 127
    assert ((s >= lo) & (s <= hi)).all()
    f = np.exp2(s.astype(np.float64) - 127)[:, :, None]
    u = np.abs(b(h)) / f
    half = np.where(u < 2, 0.25, np.where(u < 4, 0.5, 1.0)) * f
    v = b(rm.mx_values(code, s))
    # where h's own interval crosses into a wider step, that step's half
    wide = np.where(u + b(tol) / f < 2, 0.25, np.where(u + b(tol) / f < 4, 0.5, 1.0)) * f
    assert (np.abs(v - b(h)) <= np.maximum(half, wide) + b(tol) * 1.0001).all()


CASES = [
    # T, E, k, n, d, I, counts (None: a routing of distinct picks)
    (1, 1, 1, 1, 128, 128, [1]),
    (1, 8, 2, 4, 256, 128, [0, 1, 0, 1]),
    (8, 256, 8, 32, 512, 256, None),
    (5, 4, 3, 3, 128, 384, [0, 0, 0]),
    (40, 16, 4, 5, 384, 256, [0, 16, 17, 32, 33]),
    (64, 8, 8, 2, 640, 128, [64, 63]),
    (200, 8, 2, 4, 256, 384, [65, 1, 129, 200]),
    (150, 2, 2, 2, 256, 256, [150, 149]),  # tiles from here on
    (500, 8, 8, 3, 384, 640, [127, 0, 500]),
    (300, 4, 4, 4, 128, 128, [128, 129, 256, 1]),
    (1000, 32, 8, 32, 512, 256, None),
    # both tile kernels: heights on either side of each instance's, rests that join the tile in front
    (300, 8, 1, 8, 128, 384, [1, 32, 33, 64, 65, 0, 5, 100]),
    (800, 9, 1, 8, 384, 128, [127, 128, 129, 192, 193, 1, 0, 30]),
    (2000, 8, 1, 8, 256, 128, [1, 64, 65, 128, 129, 192, 193, 257]),
    (3000, 8, 1, 8, 384, 256, [256, 319, 320, 321, 0, 577, 513, 400]),
    (4000, 2, 1, 2, 128, 384, [1025, 2112]),
    (900, 3, 2, 3, 1152, 128, [300, 290, 310]),
]


def _routing(T, E, k, n, counts, seed):
    if counts is not None:
        return _counts_to_rows(counts, T, k, seed)
    r = np.random.default_rng([seed, T])
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    _, offsets, rows, _ = rm.sort_picks(ids, 0, n)
    return offsets, rows


@pytest.mark.parametrize("h_type", [mb.MOE_BF16, mb.MOE_MXFP4])
@pytest.mark.parametrize("T,E,k,n,d,I,counts", CASES)
def test_gate_up(T, E, k, n, d, I, counts, h_type):  # noqa: E741
    offsets, rows = _routing(T, E, k, n, counts, 1)
    total, R = int(offsets[-1]), T * k
    code, s = _x(T, d, 2)
    xv = rm.mx_values(code, s)
    w13, wv = _expert_weights(n, 2 * I, d, mb.MOE_W13, d, I, 3)
    mx = h_type == mb.MOE_MXFP4
    h = torch.full((R + 1, I // 2) if mx else (R + 1, I), 77, dtype=torch.uint8 if mx else torch.bfloat16, device="cuda")
    hs = torch.full((R + 1, I // 32), 77, dtype=torch.uint8, device="cuda") if mx else None
    mb.moe_mx_gate_up(_group(T, E, k, n, d, I, h_type), _cuda(rm.mx_pack(code)), _cuda(s), _cuda(offsets), _cuda(rows), w13, h,
                      hs)
    torch.cuda.synchronize()
    assert bool((h[total:] == 77).all()) and (hs is None or bool((hs[total:] == 77).all())), "wrote other rows"
    for e in range(n):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        gu, mag = rm.product(xv[rows[lo:hi]], wv[e])
        tol = rm.product_tol(mag, d)
        ref = rm.swiglu(gu[:, :I], gu[:, I:])
        t = rm.swiglu_tol(gu[:, :I], gu[:, I:], tol[:, :I], tol[:, I:])
        if mx:
            _check_h_mx(rm.mx_unpack(to_np(h[lo:hi])), to_np(hs[lo:hi]), ref, t)
        else:
            got = h[lo:hi].double().cpu().numpy()
            assert (np.abs(got - ref) <= t + (np.abs(ref) + t) * 2.0**-8).all()


@pytest.mark.parametrize("out_type", [mb.MOE_BF16, mb.MOE_FP32])
@pytest.mark.parametrize("T,E,k,n,d,I,counts", CASES)
def test_down(T, E, k, n, d, I, counts, out_type):  # noqa: E741
    offsets, _ = _routing(T, E, k, n, counts, 1)
    total, R = int(offsets[-1]), T * k
    code, s = np.zeros((R, I), np.uint8), np.full((R, I // 32), 255, np.uint8)  # rows behind the last: NaN
    code[:total], s[:total] = _x(total, I, 4) if total else (code[:0], s[:0])
    w2, wv = _expert_weights(n, d, I, mb.MOE_W2, d, I, 5)
    bf = out_type == mb.MOE_BF16
    y = torch.full((R + 1, d), 77, dtype=torch.bfloat16 if bf else torch.float32, device="cuda")
    mb.moe_mx_down(_group(T, E, k, n, d, I, out_type=out_type), _cuda(rm.mx_pack(code)), _cuda(s), _cuda(offsets), w2, y)
    torch.cuda.synchronize()
    assert bool((y[total:] == 77).all()), "wrote other rows"
    xv = rm.mx_values(code[:total], s[:total])
    for e in range(n):
        lo, hi = offsets[e], offsets[e + 1]
        ref, mag = rm.product(xv[lo:hi], wv[e])
        got = y[lo:hi].double().cpu().numpy()
        assert (np.abs(got - ref) <= rm.product_tol(mag, I) + rm.half_step("bf16" if bf else "fp32") * np.abs(ref) * 1.01).all()


# wide weights of many experts: the tiles of 256 x 256, whose last one takes up to 320 rows
MANY = [0, 1, 64, 65, 128, 129, 192, 193, 255, 256, 257, 319, 320, 321, 384, 385, 511, 512, 513, 576, 577, 40, 0, 0, 7, 100,
        31, 32, 33, 2, 0, 3]
LARGE = [
    (1000, 32, 8, 32, 128, 896, MANY),
    (1000, 32, 8, 32, 1792, 128, MANY),
    (64, 32, 8, 32, 1920, 896, None),
    (8000, 8, 1, 8, 1792, 896, [1000, 1025, 1088, 1089, 0, 1300, 1000, 1498]),
]


@pytest.mark.parametrize("h_type", [mb.MOE_BF16, mb.MOE_MXFP4])
@pytest.mark.parametrize("T,E,k,n,d,I,counts", LARGE)
def test_gate_up_of_wide_experts(T, E, k, n, d, I, counts, h_type):  # noqa: E741
    test_gate_up(T, E, k, n, d, I, counts, h_type)


@pytest.mark.parametrize("out_type", [mb.MOE_BF16, mb.MOE_FP32])
@pytest.mark.parametrize("T,E,k,n,d,I,counts", LARGE)
def test_down_of_wide_experts(T, E, k, n, d, I, counts, out_type):  # noqa: E741
    test_down(T, E, k, n, d, I, counts, out_type)


def test_gate_up_of_rows_that_are_not_finite():
    """A NaN row stays alone; its MXFP4 blocks are NaN with zero codes."""
    for T in (20, 300):
        code, s = _x(T, 256, 6)
        s[3, 1] = 255
        w13, _ = _expert_weights(1, 256, 256, mb.MOE_W13, 256, 128, 7)
        offsets, rows = np.array([0, T], np.int32), np.arange(T, dtype=np.int32)
        h = torch.empty((T, 64), dtype=torch.uint8, device="cuda")
        hs = torch.empty((T, 4), dtype=torch.uint8, device="cuda")
        mb.moe_mx_gate_up(_group(T, 1, 1, 1, 256, 128), _cuda(rm.mx_pack(code)), _cuda(s), _cuda(offsets), _cuda(rows), w13, h, hs)
        hs, h = to_np(hs), to_np(h)
        assert (hs[3] == 255).all() and not h[3].any() and (np.delete(hs, 3, axis=0) < 255).all()


def test_offsets_and_rows_outside_are_the_nearer_end():
    """Offsets behind the sorted rows and tokens outside the tokens read and write nothing
    outside the buffers."""
    T, k, d, I = 6, 2, 128, 128  # noqa: E741
    code, s = _x(T, d, 8)
    w13, _ = _expert_weights(2, 2 * I, d, mb.MOE_W13, d, I, 9)
    run = lambda off, rows, h: mb.moe_mx_gate_up(  # noqa: E731
        _group(T, 2, k, 2, d, I, mb.MOE_BF16), _cuda(rm.mx_pack(code)), _cuda(s), _cuda(np.array(off, np.int32)),
        _cuda(np.array(rows, np.int32)), w13, h)
    a = torch.full((T * k + 4, I), 77.0, dtype=torch.bfloat16, device="cuda")
    b = a.clone()
    run([0, 5, 12], [0, 5, 0, 1, 2, 3, 4, 5, 0, 5, 5, 5], a)
    run([-3, 5, 10**6], [-7, 6, 0, 1, 2, 3, 4, 5, 0, 10**9, 5, 77], b)
    assert torch.equal(a, b) and bool((b[T * k:] == 77).all())


# ------------------------------------------------------------------ the path as one


class Path:
    """One GPU's share of the layer for T rows: forward to its partial and back to the
    logits' and the rows' gradients (the experts' own backward is left out: dxs is given)."""

    def __init__(self, T, E, k, n, base, d, I, seed, balance=True):  # noqa: E741
        g = torch.Generator(device="cuda").manual_seed(seed)
        f32, i32, u8 = dict(device="cuda"), dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.uint8, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        R = T * k
        self.shape = (T, E, k, n, base, d, I)
        self.g, self.R = g, R
        self.gd = mb.gate_dims_from(dict(T=T, E=E, topk=k, score=mb.MOE_SCORE_SIGMOID, renorm=1, bias_mode=1))
        self.rd = mb.rows_dims_from(dict(T=T, E=E, topk=k, n_local=n, local_base=base, d=d, tok_type=mb.MOE_FP32,
                                         row_type=mb.MOE_BF16))
        self.xd = mb.mx_dims_from(dict(M=T, K=d, in_type=mb.MOE_BF16))
        self.md = _group(T, E, k, n, d, I)
        self.bd = mb.balance_dims_from(dict(T=T, E=E, topk=k, n_seq=1, coef=0.01))
        self.w13, self.v13 = _expert_weights(n, 2 * I, d, mb.MOE_W13, d, I, seed)
        self.w2, self.v2 = _expert_weights(n, d, I, mb.MOE_W2, d, I, seed + 1)
        self.logits, self.bias = torch.empty((T, E), **f32), torch.empty(E, **f32)
        self.x, self.dout = torch.empty((T, d), **bf), torch.empty((T, d), **f32)
        self.ids, self.w = torch.empty((T, k), **i32), torch.empty((T, k), **f32)
        self.counts, self.offsets = torch.empty(n, **i32), torch.empty(n + 1, **i32)
        self.rows, self.pos = torch.empty(R, **i32), torch.empty((T, k), **i32)
        self.xq, self.xs = torch.empty((T, d // 2), **u8), torch.empty((T, d // 32), **u8)
        self.hq, self.hs = torch.zeros((R, I // 2), **u8), torch.zeros((R, I // 32), **u8)
        self.y, self.dy = torch.zeros((R, d), **bf), torch.zeros((R, d), **bf)
        self.out, self.dw = torch.empty((T, d), **f32), torch.empty((T, k), **f32)
        self.dx = torch.empty((T, d), **f32)
        self.bcounts, self.probs = torch.empty((1, E), **i32), torch.empty((1, E), **f32)
        self.loss, self.dlogits = torch.empty(1, **f32), torch.empty((T, E), **f32)
        self.ws = torch.zeros(mb.moe_sort_workspace_bytes(self.rd), **u8)
        self.bws = torch.zeros(mb.moe_balance_workspace_bytes(self.bd), **u8)
        self.fill()

    def fill(self):
        for t in (self.logits, self.x, self.dout):
            t.normal_(generator=self.g)
        self.bias.normal_(0.0, 0.3, generator=self.g)
        self.logits[-2:] = float("-inf")  # padded rows

    def step(self, stream=None):
        k = dict(stream=stream)
        mb.moe_gate(self.gd, self.logits, self.bias, self.ids, self.w, **k)
        mb.moe_sort(self.rd, self.ids, self.counts, self.offsets, self.rows, self.pos, self.ws, **k)
        mb.moe_mx_quant(self.xd, self.x, self.xq, self.xs, **k)
        mb.moe_mx_gate_up(self.md, self.xq, self.xs, self.offsets, self.rows, self.w13, self.hq, self.hs, **k)
        mb.moe_mx_down(self.md, self.hq, self.hs, self.offsets, self.w2, self.y, **k)
        mb.moe_return(self.rd, self.y, self.w, self.pos, self.out, **k)
        mb.moe_balance_loss(self.bd, self.logits, self.ids, None, self.bcounts, self.probs, self.loss, self.bws, **k)
        mb.moe_return_backward(self.rd, self.dout, self.y, self.w, self.pos, self.dy, self.dw, **k)
        mb.moe_balance_backward(self.bd, self.logits, self.bcounts, None, None, self.dlogits, **k)
        mb.moe_gate_backward(self.gd, self.logits, self.ids, self.dw, self.dlogits, self.dlogits, **k)
        mb.moe_return(self.rd, self.dy, None, self.pos, self.dx, **k)

    OUT = ("ids", "w", "counts", "offsets", "rows", "pos", "xq", "xs", "out", "dw", "dx", "dlogits", "loss", "y", "dy", "hq", "hs")

    def result(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).clone() for k in self.OUT}


@pytest.mark.parametrize("T,E,k,n,base,d,I", [(16, 16, 4, 4, 4, 256, 128), (200, 64, 8, 16, 16, 512, 256),
                                              (700, 16, 4, 8, 8, 384, 384)])
def test_path(T, E, k, n, base, d, I):  # noqa: E741
    """Every step against its reference on the GPU's own inputs of that step."""
    p = Path(T, E, k, n, base, d, I, 1)
    p.step()
    r = {k2: v.double().cpu().numpy() if v.dtype.is_floating_point else to_np(v) for k2, v in p.result().items()}
    l, bias = to_np(p.logits), to_np(p.bias)
    ids, w = rm.gate(l, bias, k, "sigmoid", 1)
    assert np.array_equal(r["ids"], ids) and (np.abs(r["w"] - w) <= rm.gate_rel(l) * w + 1e-37).all()
    counts, offsets, rows, pos = rm.sort_picks(ids, base, n)
    for a, b in (("counts", counts), ("offsets", offsets), ("rows", rows), ("pos", pos)):
        assert np.array_equal(r[a], b)
    code, s = rm.mx_quant(p.x.double().cpu().numpy())
    assert np.array_equal(r["xs"], s)
    xv = rm.mx_values(code, s)
    total = offsets[-1]
    hc = rm.mx_unpack(r["hq"])
    hv = rm.mx_values(hc, r["hs"])
    for e in range(n):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        gu, mag = rm.product(xv[rows[lo:hi]], p.v13[e])
        tol = rm.product_tol(mag, d)
        ref = rm.swiglu(gu[:, :I], gu[:, I:])
        _check_h_mx(hc[lo:hi], r["hs"][lo:hi], ref, rm.swiglu_tol(gu[:, :I], gu[:, I:], tol[:, :I], tol[:, I:]))
        ref, mag = rm.product(hv[lo:hi], p.v2[e])
        assert (np.abs(r["y"][lo:hi] - ref) <= rm.product_tol(mag, I) + 2.0**-8 * 1.01 * np.abs(ref)).all()
    w32 = r["w"]
    ref, mag = rm.weighted_sum(r["y"], w32, pos)
    assert (np.abs(r["out"] - ref) <= (k + 1) * rm.U24 * mag).all()
    assert not r["out"][-2:].any() and not r["dx"][-2:].any() and not r["dlogits"][-2:].any()
    dout = p.dout.double().cpu().numpy()
    dw = np.zeros((T, k))
    dy = np.zeros((T * k, d))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                dw[t, j] = dout[t] @ r["y"][pos[t, j]]
                dy[pos[t, j]] = w32[t, j] * dout[t]
    assert (np.abs(r["dy"] - dy)[:total] <= 1.01 * (2.0**-8 + rm.U24) * np.abs(dy)[:total]).all()
    mags = np.zeros((T, k))
    for j in range(k):
        on = pos[:, j] >= 0
        mags[on, j] = (np.abs(dout[on]) * np.abs(r["y"][pos[on, j]])).sum(axis=1)
    assert (np.abs(r["dw"] - dw) <= (8 * -(-d // 128) + 10) * rm.U24 * mags).all()
    grad, gmag = rm.gate_grad(l, ids, r["dw"], "sigmoid", 1)
    from tests._ref_fp8 import balance

    bal = np.nan_to_num(balance(l.astype(np.float64), ids, [0, T], 1, "sigmoid", 0.01)[3])
    tol = (rm.gate_rel(l) * 2 + 20 * rm.U24) * gmag + 1e-4 * np.abs(bal).max() * 2.0**-8 + rm.U24 * 2 * np.abs(grad + bal)
    assert (np.abs(r["dlogits"] - grad - bal) <= tol).all()


def test_path_in_a_graph():
    """Captured once, replayed on new inputs, with eager work and synchronizations between."""
    p = Path(300, 32, 4, 8, 8, 256, 256, 2)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        p.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        p.step()
    for i in range(4):
        p.fill()
        p.step()
        want = p.result()
        for key in p.OUT:  # what the replay has to write again
            if key not in ("y", "dy", "hq", "hs"):
                getattr(p, key).zero_()
        torch.cuda.synchronize()
        graph.replay()
        got = p.result()
        for key in p.OUT:
            assert torch.equal(got[key], want[key]), (i, key)


def test_two_paths_on_two_streams():
    paths = [Path(250, 32, 4, 8, 8, 256, 256, 3), Path(190, 32, 8, 16, 0, 384, 128, 4)]
    want = []
    for p in paths:
        p.step()
        want.append(p.result())
    streams = [torch.cuda.Stream() for _ in paths]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, st in zip(paths, streams):
            p.step(st)
    for p, ref in zip(paths, want):
        got = p.result()
        assert all(torch.equal(got[key], ref[key]) for key in p.OUT)


def test_path_repeats_bit_for_bit():
    p = Path(1500, 64, 8, 32, 0, 512, 256, 5)
    p.step()
    want = p.result()
    for _ in range(3):
        p.step()
        got = p.result()
        assert all(torch.equal(got[key], want[key]) for key in p.OUT)


def test_experts_of_a_graph_replayed():
    """The kernels of wide experts and of one expert's few rows, captured and replayed on other
    offsets and rows than they were captured with."""
    for T, E, k, n, d, I, all_counts in (  # noqa: E741
        (1000, 32, 8, 32, 1792, 896, [MANY, MANY[::-1], [0] * 32, [8000] + [0] * 31]),
        (20, 8, 2, 2, 256, 128, [[20, 20], [0, 1], [0, 0], [17, 0]]),
    ):
        md = _group(T, E, k, n, d, I)
        w13, _ = _expert_weights(n, 2 * I, d, mb.MOE_W13, d, I, 5)
        w2, _ = _expert_weights(n, d, I, mb.MOE_W2, d, I, 6)
        code, sc = _x(T, d, 7)
        xq, xs = _cuda(rm.mx_pack(code)), _cuda(sc)
        R = T * k
        off, rows = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
        hq = torch.zeros((R, I // 2), dtype=torch.uint8, device="cuda")
        hs = torch.zeros((R, I // 32), dtype=torch.uint8, device="cuda")
        y = torch.zeros((R, d), dtype=torch.bfloat16, device="cuda")

        def step(stream=None):
            mb.moe_mx_gate_up(md, xq, xs, off, rows, w13, hq, hs, stream=stream)
            mb.moe_mx_down(md, hq, hs, off, w2, y, stream=stream)

        def put(i):
            o, r = _counts_to_rows(all_counts[i], T, k, i)
            off.copy_(torch.from_numpy(o))
            rows.copy_(torch.from_numpy(r))
            for t in (hq, hs, y):
                t.zero_()

        stream = torch.cuda.Stream()
        put(0)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for i in (1, 0, 2, 3, 0):
            put(i)
            step()
            want = [t.clone() for t in (hq, hs, y)]
            put(i)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((hq, hs, y), want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (T, i)
