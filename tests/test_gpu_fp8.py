"""GPU parity of the FP8 (block-128) calls against the 64-bit references of
tests/_ref_fp8.py (which derives the tolerances): moe_fp8_quant bit for bit,
moe_fp8_gemm / moe_fp8_proj and moe_fp8_expert_ffn within the bound of an fp32
accumulation plus one rounding of the output."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
import oracle  # noqa: E402
from synth import get_config, make_fp8_inputs, make_fp8_weight  # noqa: E402
from tests import _ref_fp8 as rf  # noqa: E402
from tests._ref import bf16_val  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402

KIND = {"bf16": mb.MOE_BF16, "fp32": mb.MOE_FP32}
TT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rows(M, K, kind, seed):
    r = np.random.default_rng([seed, M, K])
    x = r.standard_normal((M, K)) * np.exp(r.standard_normal((M, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(TT[kind])


def _guarded(shape, dtype, fill):
    """A tensor inside a larger buffer whose bytes behind it hold `fill`."""
    n = int(np.prod(shape))
    size = torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n * size + 4096,), fill, dtype=torch.uint8, device="cuda")
    return raw[:n * size].view(dtype).view(shape), raw[n * size:]


def _quant(x, dims):
    kb = -(-dims.K // 128)
    xq, g1 = _guarded((dims.M, kb * 128), torch.uint8, 0xA5)
    xs, g2 = _guarded((kb, dims.M), torch.float32, 0xA5)
    mb.moe_fp8_quant(dims, x, xq, xs)
    torch.cuda.synchronize()
    assert bool((g1 == 0xA5).all()) and bool((g2 == 0xA5).all()), "wrote behind its outputs"
    return xq, xs


def _check_quant(x, dims):
    xq, xs = _quant(x.cuda(), dims)
    q, s = rf.quant(x.double().numpy())
    got_s = to_np(xs).astype(np.float64)
    assert np.array_equal(got_s, s, equal_nan=True)
    a, b = rf.TABLE[to_np(xq)], rf.TABLE[q]
    assert np.array_equal(a, b, equal_nan=True)
    assert np.array_equal(np.signbit(a[~np.isnan(a)]), np.signbit(b[~np.isnan(b)]))


# ------------------------------------------------------------------ quantise


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (2, 127), (3, 129), (16, 1000), (5, 130), (77, 2120), (300, 4096),
                                 (1, 32768), (2000, 36)])
def test_quant(M, K, kind):
    _check_quant(_rows(M, K, kind, 0), mb.fp8_dims_from(dict(M=M, K=K, in_type=KIND[kind])))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_quant_edge_values(kind):
    x = _rows(12, 300, kind, 1)
    big = torch.finfo(TT[kind]).max
    x[0] = 0
    x[1] = 1e-39
    x[2, :140] = 448.0
    x[3, 5] = float("inf")
    x[4, 200] = float("nan")
    x[5, 299] = -float("inf")
    x[6, 0], x[6, 1] = big, -big
    x[7, :128] = torch.from_numpy(np.concatenate([rf._MID, [448.0, -448.0]]).astype(np.float32)).to(TT[kind])
    x[8] = -0.0
    x[9] = 2.0**-126
    x[10, 3] = 449.0
    _check_quant(x, mb.fp8_dims_from(dict(M=12, K=300, in_type=KIND[kind])))


# ------------------------------------------------------------------ product


def _product(dims, x, q, s):
    """proj, and quant + gemm on a poisoned output: the same bits."""
    packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    kind = "bf16" if dims.out_type == mb.MOE_BF16 else "fp32"
    out, guard = _guarded((dims.M, dims.N), TT[kind], 0x7F)
    ws = torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    xg = x.cuda()
    mb.moe_fp8_proj(dims, xg, packed, out, ws)
    out2, guard2 = _guarded((dims.M, dims.N), TT[kind], 0x7F)
    gws = torch.zeros(mb.moe_fp8_gemm_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    xq, xs = _quant(xg, dims)
    mb.moe_fp8_gemm(dims, xq, xs, packed, out2, gws)
    first = out.clone()
    mb.moe_fp8_proj(dims, xg, packed, out, ws)  # the workspaces are ready again
    mb.moe_fp8_gemm(dims, xq, xs, packed, out2, gws)
    torch.cuda.synchronize()
    assert bool((guard == 0x7F).all()) and bool((guard2 == 0x7F).all()), "wrote behind its output"
    assert torch.equal(first, out) and torch.equal(out, out2)
    return out.double().cpu().numpy(), kind


def _check_product(M, N, K, kind_in, kind_out, seed=0):
    dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, in_type=KIND[kind_in], out_type=KIND[kind_out]))
    x = _rows(M, K, kind_in, seed)
    q, s = make_fp8_weight((N, K), seed)
    got, _ = _product(dims, x, q, s)
    xv = rf.values(*rf.quant(x.double().numpy()))
    ref, mag = rf.product(xv, rf.weight(q, s))
    tol = rf.product_tol(mag, K)
    tol = tol + rf.half_step(kind_out) * (np.abs(ref) + tol)
    err = np.abs(got - ref)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), (worst, got[worst], ref[worst], tol[worst])


PRODUCTS = [
    (1, 1, 1), (1, 16, 128), (1, 4096, 1024), (2, 100, 300), (7, 63, 129), (15, 65, 2120), (16, 64, 4096), (17, 128, 640),
    (31, 257, 896), (33, 1000, 1024), (64, 512, 2048), (65, 129, 385), (77, 515, 2120), (127, 128, 512), (128, 192, 7168),
    (129, 256, 1024), (200, 384, 256), (255, 513, 1152), (256, 256, 128), (257, 300, 1300), (513, 640, 640),
    (1024, 768, 1024), (1, 33, 16384), (4, 32768, 128), (3000, 17, 64),
]


@pytest.mark.parametrize("kind_out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, kind_out):
    _check_product(M, N, K, "bf16", kind_out)


# further kernels and K splits: 64-row register tiles, LDS tiles of 128 with one,
# two and many K blocks, split and whole, tiles of 256, rows too many to quantise
# in the product, 64 weight rows a workgroup at few rows
FORMS = [
    (16, 4096, 8192), (16, 8200, 640), (3, 300, 20000), (20, 8300, 384), (64, 8300, 640), (100, 5000, 700),
    (1000, 4096, 100), (1000, 4096, 256), (700, 2000, 2100), (1500, 2100, 640), (3900, 4000, 300), (4096, 4096, 130),
    (300, 300, 300), (640, 64, 4096),
]


@pytest.mark.parametrize("kind_out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_product_forms(M, N, K, kind_out):
    _check_product(M, N, K, "bf16", kind_out, seed=1)


@pytest.mark.parametrize("M,N,K", [(1, 512, 512), (8, 1024, 4096), (100, 99, 333), (300, 256, 260)])
def test_product_from_fp32_rows(M, N, K):
    _check_product(M, N, K, "fp32", "fp32", seed=3)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_takes_any_scales(M):
    """Rows quantised elsewhere: scales that are no powers of two, zero,
    negative, of very different size; weight scales likewise."""
    N, K = 200, 1000
    r = np.random.default_rng(M)
    dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32))
    kb = 8
    xq = r.integers(0, 256, (M, kb * 128), dtype=np.uint8)
    xq[(xq & 127) == 127] = 0
    xq[:, K:] = 0
    xs = (r.standard_normal((kb, M)) * np.exp(3 * r.standard_normal((kb, M)))).astype(np.float32)
    xs[1] = 0
    q, s = make_fp8_weight((N, K), 5)
    s *= np.exp(2 * r.standard_normal(s.shape)).astype(np.float32) * np.sign(r.standard_normal(s.shape)).astype(np.float32)
    packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    out = torch.empty((M, N), device="cuda")
    ws = torch.zeros(mb.moe_fp8_gemm_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_fp8_gemm(dims, torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), packed, out, ws)
    ref, mag = rf.product(rf.values(xq, xs.astype(np.float64)), rf.weight(q, s))
    assert np.all(np.abs(to_np(out) - ref) <= rf.product_tol(mag, K) + rf.U24 * np.abs(ref))


@pytest.mark.parametrize("M", [2, 70, 300])
def test_product_of_values_that_are_not_finite(M):
    """A NaN weight spoils its output column, a row's block that is not finite
    its row; everything else is untouched."""
    N, K = 130, 384
    dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32))
    x = _rows(M, K, "bf16", 2)
    x[1, 200] = float("inf")
    q, s = make_fp8_weight((N, K), 2)
    q[129, 5] = 0xFF
    got, _ = _product_nan(dims, x, q, s)
    bad = np.zeros((M, N), bool)
    bad[1] = True
    bad[:, 129] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def _product_nan(dims, x, q, s):
    packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    out = torch.empty((dims.M, dims.N), device="cuda")
    ws = torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_fp8_proj(dims, x.cuda(), packed, out, ws)
    return out.double().cpu().numpy(), "fp32"


def test_quant_offsets_past_32_bits():
    """Rows behind 2^32 elements: the same bits as a call on those rows alone."""
    M, K, n = 135000, 32768, 40
    r = torch.Generator(device="cuda").manual_seed(5)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-n:] = torch.randn((n, K), generator=r, device="cuda").to(torch.bfloat16)
    xq = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    xs = torch.empty((K // 128, M), dtype=torch.float32, device="cuda")
    mb.moe_fp8_quant(dict(M=M, K=K), x, xq, xs)
    q1 = torch.empty((n, K), dtype=torch.uint8, device="cuda")
    s1 = torch.empty((K // 128, n), dtype=torch.float32, device="cuda")
    mb.moe_fp8_quant(dict(M=n, K=K), x[-n:].clone(), q1, s1)
    assert torch.equal(xq[-n:], q1) and torch.equal(xs[:, -n:], s1)
    assert not bool(xq[:-n].any())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product_offsets_past_32_bits(out):
    """Outputs behind 2^32 elements. One K block: every kernel form sums it alike
    for one output type from 17 rows on, so the bits are those of a call on
    the last rows alone."""
    M, N, K, n = 262144, 16500, 100, 77
    r = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((M, K), generator=r, device="cuda").to(torch.bfloat16)
    q = torch.randn((N, K), generator=r, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.rand((-(-N // 128), 1), generator=r, device="cuda") + 0.5
    kind = mb.MOE_BF16 if out == torch.bfloat16 else mb.MOE_FP32
    big = dict(M=M, N=N, K=K, out_type=kind)
    w = torch.empty(mb.moe_packed_fp8_bytes(big), dtype=torch.uint8, device="cuda")
    mb.moe_pack_fp8(big, q, sc, w)

    def run(dims, rows):
        ws = torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
        o = torch.empty((dims["M"], N), dtype=out, device="cuda")
        mb.moe_fp8_proj(dims, rows, w, o, ws)
        return o

    got = run(big, x)
    want = run(dict(big, M=n), x[-n:].clone())
    assert bool(want.abs().max() > 1)
    assert torch.equal(got[-n:], want)


def test_one_workspace_serves_other_dims():
    """The gemm workspace is left ready for any dims it is large enough for."""
    sizes = [(8, 1024, 4096), (1, 512, 8192), (100, 256, 2048), (8, 64, 16384), (400, 512, 640)]
    cases = []
    for M, N, K in sizes:
        dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32))
        q, s = make_fp8_weight((N, K), M)
        packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
        mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
        x = _rows(M, K, "bf16", 4).cuda()
        own = torch.empty((M, N), device="cuda")
        mb.moe_fp8_proj(dims, x, packed, own,
                        torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda"))
        cases.append((dims, x, packed, own))
    n = max(mb.moe_fp8_proj_workspace_bytes(c[0]) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for dims, x, packed, own in cases:
            out = torch.full_like(own, float("nan"))
            mb.moe_fp8_proj(dims, x, packed, out, ws)
            torch.cuda.synchronize()
            assert torch.equal(out, own), (dims.M, dims.N, dims.K)


# ------------------------------------------------------------------ experts


def _check_experts(cfg, seed, ids=None):
    """moe_bucket -> moe_fp8_expert_ffn on given (or routed) picks, against the
    reference on the GPU's own buckets; rows without a pick stay as they were."""
    from moe_decode_layer_router_amd.block import Fp8Block

    inp = make_fp8_inputs(cfg, seed, gamma="random")
    blk = Fp8Block(inp)
    blk.route()
    if ids is not None:
        blk.ids.copy_(torch.from_numpy(ids.astype(np.int32)))
    blk.bucket()
    blk.y.fill_(7.0)
    blk.expert_ffn()
    first = blk.y.clone()
    blk.y.fill_(7.0)
    blk.expert_ffn()
    torch.cuda.synchronize()
    assert torch.equal(first, blk.y), "two calls differ"
    y = bf16_val(to_np(blk.y))
    offsets, rows = to_np(blk.offsets), to_np(blk.rows)
    R = blk.dims.r_max
    assert np.all(y[offsets[-1]:R] == 7.0), "rows without a pick were written"
    xv = rf.values(*rf.quant(bf16_val(inp["x"])))
    jobs = [(xv[rows[offsets[e]:offsets[e + 1]]], y[offsets[e]:offsets[e + 1]],
             rf.weight(inp["w13"][0][e], inp["w13"][1][e]), rf.weight(inp["w2"][0][e], inp["w2"][1][e]), f"expert {e}")
            for e in range(cfg.n_local) if offsets[e + 1] > offsets[e]]
    if cfg.shared_I:
        jobs.append((xv, y[R:], rf.weight(*inp["ws13"]), rf.weight(*inp["ws2"]), "shared"))
    for x, got, w13, w2, what in jobs:
        ref, tol = rf.ffn_row_tol(x, w13, w2)
        tol = tol + rf.half_step("bf16") * (np.abs(ref) + tol)
        err = np.abs(got - ref)
        assert np.all(err <= tol), (what, float((err / tol).max()))
        # the moves of h across rounding borders are rare: in the 2-norm the
        # output's own rounding (at most half a step a value) is what is left
        assert np.linalg.norm(got - ref) <= (rf.half_step("bf16") + 1e-4) * np.linalg.norm(ref), what
    return blk, inp


SMALL = get_config("tiny")
EXPERTS = {
    "tiny": SMALL,
    "S16_many_blocks": SMALL.with_(S=16, d=4608, I=256),  # 576 (row, K block) pairs: still quantised in place
    "S16_too_many_blocks": SMALL.with_(S=16, d=4736, I=256),
    "S17": SMALL.with_(S=17, E=2, n_local=2, topk=2),  # two token tiles a bucket
    "shared_wider_than_I": SMALL.with_(S=9, I=128, shared_I=1024),
    "S1": SMALL.with_(S=1),
    "S1_top8": SMALL.with_(S=1, topk=8),
    "one_expert_64_rows": SMALL.with_(S=64, E=1, n_local=1, topk=1),
    "one_expert_128_rows": SMALL.with_(S=128, E=1, n_local=1, topk=1),
    "ragged_buckets": SMALL.with_(S=100, E=9, n_local=5, local_base=3, topk=4, I=384, d=640),
    "not_all_local": SMALL.with_(S=16, E=64, n_local=8, local_base=56, topk=8),
    "shared": SMALL.with_(S=40, shared_I=256, d=512),
    "shared_S1": SMALL.with_(S=1, shared_I=128),
    "shared_S128": SMALL.with_(S=128, E=32, n_local=4, topk=8, shared_I=384, I=256, d=384),
    "wide": SMALL.with_(S=5, d=4096, I=128),
    "long_I": SMALL.with_(S=5, d=128, I=2048, shared_I=1024),
}


@pytest.mark.parametrize("name", list(EXPERTS))
def test_experts(name):
    _check_experts(EXPERTS[name], 11)


def test_experts_without_a_local_pick():
    cfg = SMALL.with_(S=8, E=16, n_local=4, local_base=4, topk=2)
    ids = np.tile([0, 15], (8, 1))
    _check_experts(cfg, 1, ids)
    _check_experts(cfg.with_(shared_I=128), 1, ids)


def test_experts_uneven_buckets():
    """All rows on one expert, one row on another, the rest empty."""
    cfg = SMALL.with_(S=90, E=8, n_local=8, topk=2)
    ids = np.tile([3, 100], (90, 1))  # the second pick is held elsewhere
    ids[17, 1] = 6
    _check_experts(cfg, 2, ids)


def test_workload_s8():
    _check_experts(get_config("s8_uniform").with_(n_local=8, local_base=0, E=64, I=512), 0)


def test_block_chain_with_counts():
    """route -> bucket -> FP8 experts -> combine, as a decode step runs them,
    and the step's per-expert counts and balance loss from its routing."""
    cfg = SMALL.with_(S=48, E=32, n_local=16, local_base=8, topk=4, shared_I=256, bias_mode=0)
    blk, inp = _check_experts(cfg, 21)
    blk.step()
    bal = mb.balance_dims_from(dict(T=cfg.S, E=cfg.E, topk=cfg.topk, n_seq=1, coef=0.01))
    ws = torch.zeros(mb.moe_balance_workspace_bytes(bal), dtype=torch.uint8, device="cuda")
    counts = torch.empty((1, cfg.E), dtype=torch.int32, device="cuda")
    probs = torch.empty((1, cfg.E), device="cuda")
    loss = torch.empty(1, device="cuda")
    mb.moe_balance_loss(bal, blk.logits, blk.ids, None, counts, probs, loss, ws)
    torch.cuda.synchronize()
    ids, w = to_np(blk.ids), to_np(blk.w)
    lo = oracle.router_logits(inp["x"], inp["wr"], inp["bias"])
    want_ids, want_w = oracle.topk(lo, cfg.topk, cfg.renorm)
    assert np.array_equal(ids, want_ids)
    out = oracle.combine(cfg, to_np(blk.y), w, to_np(blk.pick_pos), inp["gamma"])
    rms = np.sqrt(np.mean(out.astype(np.float64) ** 2))
    assert np.abs(to_np(blk.out) - out).max() <= 2e-2 * rms
    assert np.array_equal(to_np(counts)[0], np.bincount(ids.reshape(-1), minlength=cfg.E))
    assert np.array_equal(to_np(counts)[0, 8:24], to_np(blk.counts))
    ref = rf.balance(to_np(blk.logits), ids, [0, cfg.S], 1, "sigmoid", 0.01)
    assert abs(float(loss) - ref[2]) <= 64 * rf.U24 * ref[2]


# ------------------------------------------------------------------ streams, graphs, refusals


def _proj_case(M=8, N=512, K=2048, seed=0):
    dims = mb.fp8_dims_from(dict(M=M, N=N, K=K))
    q, s = make_fp8_weight((N, K), seed)
    packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    x = _rows(M, K, "bf16", seed).cuda()
    ws = torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    return dims, x, packed, torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), ws


@pytest.mark.parametrize("M,N", [(1, 512), (8, 512), (100, 512), (400, 512), (700, 2000)])
def test_graph_replays_match_eager(M, N):
    """Two captured graphs share a workspace and take turns with eager calls."""
    dims, x, packed, out, ws = _proj_case(M=M, N=N)
    mb.moe_fp8_proj(dims, x, packed, out, ws)
    torch.cuda.synchronize()
    ref = out.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            mb.moe_fp8_proj(dims, x, packed, out, ws)
        graphs.append(g)
    for i in range(4):
        out.fill_(float("nan"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), i
        out.fill_(float("nan"))
        mb.moe_fp8_proj(dims, x, packed, out, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), (i, "eager")


@pytest.mark.parametrize("name", ["tiny", "shared"])
def test_block_graph_replays_match_eager(name):
    from moe_decode_layer_router_amd.block import Fp8Block

    blk = Fp8Block(make_fp8_inputs(EXPERTS[name], 5))
    blk.step()
    torch.cuda.synchronize()
    ref = blk.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        blk.step()
    for i in range(3):
        blk.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(blk.out, ref), i
        blk.step()
        torch.cuda.synchronize()
        assert torch.equal(blk.out, ref), (i, "eager")


def test_experts_two_streams_and_shared_weights():
    """Two blocks on the same packed weights, buckets of their own, on two
    streams at once."""
    from moe_decode_layer_router_amd.block import Fp8Block

    inp = make_fp8_inputs(EXPERTS["shared"], 8)
    blocks = [Fp8Block(inp), Fp8Block(inp)]
    blocks[1].x.copy_(-blocks[1].x)
    blocks[1].packed = blocks[0].packed
    refs = []
    for b in blocks:
        b.step()
        refs.append(b.out.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(10):
        for st, b in zip(streams, blocks):
            with torch.cuda.stream(st):
                b.expert_ffn()
                b.combine()
    torch.cuda.synchronize()
    for b, ref in zip(blocks, refs):
        assert torch.equal(b.out, ref)


def test_two_streams_with_their_own_workspaces():
    cases = [_proj_case(M=8, N=1024, K=4096, seed=1), _proj_case(M=8, N=1024, K=4096, seed=2)]
    refs = []
    for dims, x, packed, out, ws in cases:
        mb.moe_fp8_proj(dims, x, packed, out, ws)
        refs.append(out.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for st, (dims, x, packed, out, ws) in zip(streams, cases):
            mb.moe_fp8_proj(dims, x, packed, out, ws, stream=st)
    torch.cuda.synchronize()
    for (_, _, _, out, _), ref in zip(cases, refs):
        assert torch.equal(out, ref)


def test_binding_refuses():
    dims, x, packed, out, ws = _proj_case()
    bad = [
        (x[:, ::2], packed, out, ws),  # not contiguous
        (x.cpu(), packed, out, ws),  # not on the GPU
        (x.float(), packed, out, ws),  # not in_type
        (x[:4], packed, out, ws),  # too small
        (x, packed, out[:, :100].contiguous(), ws),
        (x, packed[:1000], out, ws),
        (x, packed, out.float(), ws),
    ]
    for a in bad:
        with pytest.raises(ValueError):
            mb.moe_fp8_proj(dims, *a)
    with pytest.raises(mb.MoeError) as e:
        mb.moe_fp8_proj(dims, x, packed, out, ws[:256])
    assert e.value.code == mb.MOE_ERR_WORKSPACE
    with pytest.raises(mb.MoeError) as e:
        mb.moe_fp8_proj(dict(M=0, N=5, K=7), x, packed, out, ws)
    assert e.value.code == mb.MOE_ERR_SHAPE
