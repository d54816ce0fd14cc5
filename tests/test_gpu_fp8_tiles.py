"""The FP8 products' LDS tile kernels over many K blocks, any scales and values that are
not finite; fp32 rows into bf16 outputs; the experts at full width. Every case says
which kernel it is for (tests/_fp8_plan.py); tolerances as in test_gpu_fp8_sums.py."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_decode_layer_router_amd as mb  # noqa: E402
from synth import get_config, make_fp8_inputs, make_fp8_weight  # noqa: E402
from tests import _ref_fp8 as rf  # noqa: E402
from tests._fp8_plan import plan  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402
from tests.test_gpu_fp8_sums import KIND, TT, _check, fast_tol  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# M, N, K, outputs, form, K parts: 2 to 17 K blocks a part (the weights' three and the
# rows' two buffers come round several times), last blocks that are not whole, rows and
# columns that end inside a tile
TILES = [
    (3900, 4000, 1300, "bf16", "tile256", 1), (4096, 4096, 896, "bf16", "tile256", 1), (3841, 3900, 520, "bf16", "tile256", 1),
    (3900, 4000, 1300, "fp32", "tile128", 1), (1500, 2100, 1290, "fp32", "tile128", 1), (1500, 2100, 1290, "bf16", "tile128", 1),
    (2048, 4096, 392, "bf16", "tile128", 1), (700, 2000, 2100, "bf16", "tile128", 2), (700, 2000, 2100, "fp32", "tile128", 2),
    (513, 2700, 3500, "bf16", "tile128", 2), (330, 4096, 4200, "fp32", "tile128", 2), (1000, 1500, 4001, "fp32", "tile128", 2),
    (25000, 17, 300, "bf16", "tile128", 1), (25000, 17, 300, "fp32", "tile128", 1), (25000, 1, 129, "bf16", "tile128", 1),
    (6500, 256, 3400, "bf16", "tile128", 2), (1300, 1100, 4000, "bf16", "tile128", 2),
]


def _rows(M, K, seed):
    """e4m3 rows [M, Kp] with zeros from column K on, and power-of-two scales."""
    r = np.random.default_rng([seed, M, K])
    kb = -(-K // 128)
    xq = np.zeros((M, kb * 128), np.uint8)
    v = np.clip(r.standard_normal((M, K)) * 110.0, -448, 448)
    xq[:, :K] = rf.e4m3_encode(v)
    return xq, np.exp2(r.integers(-9, -5, (kb, M))).astype(np.float32)


@pytest.mark.parametrize("M,N,K,kind,form,parts", TILES)
def test_tiles(M, N, K, kind, form, parts):
    p = plan(M, N, K, kind)
    assert (p.form, p.parts) == (form, parts)
    xq, xs = _rows(M, K, 1)
    q, s = make_fp8_weight((N, K), 1)
    _check(M, N, K, kind, xq, xs, q, s)


FORMS = [
    (3900, 4000, 700, "bf16", "tile256"), (1300, 2100, 700, "bf16", "tile128"), (700, 2000, 2100, "bf16", "tile128"),
    (1300, 2100, 700, "fp32", "tile128"), (700, 2000, 2100, "fp32", "tile128"), (300, 200, 1000, "bf16", "mid"),
    (100, 200, 1000, "bf16", "mid"), (20, 200, 1000, "bf16", "mid"), (9, 200, 1000, "bf16", "rows"),
]


@pytest.mark.parametrize("M,N,K,kind,form", FORMS)
def test_any_scales(M, N, K, kind, form):
    """Scales that are no powers of two, zero, negative, of very different size."""
    assert plan(M, N, K, kind).form == form
    r = np.random.default_rng(M)
    kb = -(-K // 128)
    xq = r.integers(0, 256, (M, kb * 128), dtype=np.uint8)
    xq[(xq & 127) == 127] = 0
    xq[:, K:] = 0
    xs = (r.standard_normal((kb, M)) * np.exp(3 * r.standard_normal((kb, M)))).astype(np.float32)
    xs[1] = 0
    q, s = make_fp8_weight((N, K), 5)
    s *= np.exp(2 * r.standard_normal(s.shape)).astype(np.float32) * np.sign(r.standard_normal(s.shape)).astype(np.float32)
    _check(M, N, K, kind, xq, xs, q, s)


@pytest.mark.parametrize("M,N,K,kind,form", FORMS)
def test_values_that_are_not_finite(M, N, K, kind, form):
    """A NaN weight spoils its output column, a row's block that is not finite its row;
    everything else is as without them."""
    assert plan(M, N, K, kind).form == form
    dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, out_type=KIND[kind]))
    r = np.random.default_rng(M)
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    q, s = make_fp8_weight((N, K), 2)
    ws = torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")

    def run():
        mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
        out = torch.zeros((M, N), dtype=TT[kind], device="cuda")
        mb.moe_fp8_proj(dims, x, packed, out, ws)
        return out

    clean = run()
    assert bool(torch.isfinite(clean).all())
    x[1, 600] = float("inf")
    x[M - 1, K - 1] = float("nan")
    q[N - 1, 5] = 0xFF
    q[130, K - 1] = 0x7F
    got = run()
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[1] = bad[M - 1] = True
    bad[:, N - 1] = bad[:, 130] = True
    assert bool(torch.isnan(got[bad]).all())
    assert torch.equal(got[~bad], clean[~bad])


def test_one_workspace_serves_split_tiles_and_other_kernels():
    """Calls of every kernel and both kinds of outputs take turns on one workspace."""
    sizes = [(700, 2000, 2100, "bf16", "tile128", 2), (8, 1024, 4096, "bf16", "rows", 2), (700, 2000, 2100, "fp32", "tile128", 2),
             (100, 256, 2048, "bf16", "mid", 2), (513, 2700, 3500, "bf16", "tile128", 2), (3900, 4000, 300, "bf16", "tile256", 1)]
    cases = []
    for M, N, K, kind, form, parts in sizes:
        p = plan(M, N, K, kind)
        assert (p.form, p.parts) == (form, parts), (M, N, K)
        dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, out_type=KIND[kind]))
        q, s = make_fp8_weight((N, K), M)
        packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
        mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
        r = np.random.default_rng(M)
        x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
        own = torch.empty((M, N), dtype=TT[kind], device="cuda")
        mb.moe_fp8_proj(dims, x, packed, own,
                        torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda"))
        cases.append((dims, x, packed, own))
    ws = torch.zeros(max(mb.moe_fp8_proj_workspace_bytes(c[0]) for c in cases), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for dims, x, packed, own in cases:
            out = torch.full_like(own, float("nan"))
            mb.moe_fp8_proj(dims, x, packed, out, ws)
            torch.cuda.synchronize()
            assert torch.equal(out, own), (dims.M, dims.N, dims.K)


@pytest.mark.parametrize("M,N,K,form", [
    (1, 512, 512, "rows"), (8, 1024, 4096, "rows"), (16, 4096, 7168, "rows"), (16, 300, 32000, "rows"), (20, 99, 333, "mid"),
    (100, 99, 333, "mid"), (300, 256, 260, "mid"), (1300, 2100, 700, "tile128"), (3900, 4000, 300, "tile256"),
])
def test_fp32_rows_to_bf16(M, N, K, form):
    """moe_fp8_proj of fp32 rows into bf16, and the same bits from quantise and product."""
    assert plan(M, N, K, "bf16").form == form
    dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, in_type=mb.MOE_FP32))
    r = np.random.default_rng([M, N, K])
    x = (r.standard_normal((M, K)) * np.exp(r.standard_normal((M, 1)))).astype(np.float32)
    q, s = make_fp8_weight((N, K), 3)
    packed = torch.empty(mb.moe_packed_fp8_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_fp8(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mb.moe_fp8_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    xg = torch.from_numpy(x).cuda()
    mb.moe_fp8_proj(dims, xg, packed, out, ws)
    kb = -(-K // 128)
    xq = torch.empty((M, kb * 128), dtype=torch.uint8, device="cuda")
    xs = torch.empty((kb, M), device="cuda")
    mb.moe_fp8_quant(dims, xg, xq, xs)
    two = torch.empty_like(out)
    mb.moe_fp8_gemm(dims, xq, xs, packed, two, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, two)
    rq, rs = rf.quant(x.astype(np.float64))
    ref, mag = rf.product(rf.values(rq, rs), rf.weight(q, s))
    tol = rf.product_tol(mag, K)
    if not plan(M, N, K, "bf16").exact:
        tol += fast_tol(rq, rs, q, s.astype(np.float64))
    tol += rf.half_step("bf16") * (np.abs(ref) + tol)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("S,d,I,Is,E", [(8, 4096, 2048, 0, 256), (128, 7168, 2048, 2048, 256), (128, 4096, 2048, 0, 32)])
def test_experts_at_full_width(S, d, I, Is, E):  # noqa: E741
    """32 experts of the served sizes: the first, the fullest and the last with rows, and
    the shared one's last rows, against the 64-bit reference."""
    n, topk = 32, 8
    g = torch.Generator(device="cuda").manual_seed(S + d)
    dims = mb.dims_from(dict(S=S, d=d, E=E, topk=topk, n_local=n, local_base=0, I=I, renorm=1, eps=1e-6, shared_I=Is))
    w, p = {}, {}
    for key, which, shape in (("w13", mb.MOE_W13, (n, 2 * I, d)), ("w2", mb.MOE_W2, (n, d, I)),
                              ("ws13", mb.MOE_WS13, (1, 2 * Is, d)), ("ws2", mb.MOE_WS2, (1, d, Is))):
        p[key] = None
        if 0 in shape:
            continue
        q = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for m in q:
            v = (torch.randn(m.shape, generator=g, device="cuda") * 110.0).clamp_(-448, 448)
            m.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
        s = 1.8e-4 * (0.7 + 0.6 * torch.rand((shape[0], shape[1] // 128, shape[2] // 128), generator=g, device="cuda"))
        w[key] = (q, s)
        p[key] = torch.empty(mb.moe_packed_fp8_expert_bytes(dims, which), dtype=torch.uint8, device="cuda")
        mb.moe_pack_fp8_expert(dims, which, q, s, p[key])
    x = torch.randn((S, d), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand((S, E), generator=g, device="cuda").topk(topk, dim=1).indices.to(torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    R = dims.r_max
    counts, offsets, rows = torch.empty(n, **i32), torch.empty(n + 1, **i32), torch.empty(R, **i32)
    pos, active = torch.empty((S, topk), **i32), torch.empty(n + 1, **i32)
    mb.moe_bucket(dims, ids, counts, offsets, rows, pos, active)
    y = torch.full((R + (S if Is else 0), d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mb.moe_fp8_ffn_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_fp8_expert_ffn(dims, x, p["w13"], p["w2"], counts, offsets, rows, active, p["ws13"], p["ws2"], y, ws)
    torch.cuda.synchronize()
    c, o, t = to_np(counts), to_np(offsets), to_np(rows)
    used = int(o[-1])
    assert bool((y[used:R] == 7.0).all())
    full = np.nonzero(c)[0]
    jobs = [(t[o[e]:o[e + 1]], y[o[e]:o[e + 1]], e, "w13", "w2") for e in sorted({full[0], full[-1], int(c.argmax())})]
    if Is:
        jobs.append((np.arange(S - 8, S), y[-8:], 0, "ws13", "ws2"))
    for tokens, got, e, k13, k2 in jobs:
        xv = rf.values(*rf.quant(x[torch.from_numpy(tokens).long().cuda()].double().cpu().numpy()))
        mats = [rf.weight(to_np(w[k][0][e]), to_np(w[k][1][e])) for k in (k13, k2)]
        ref, tol = rf.ffn_row_tol(xv, *mats)
        err = np.abs(got.double().cpu().numpy() - ref)
        tol = tol + rf.half_step("bf16") * (np.abs(ref) + tol)
        assert np.all(err <= tol), (k13, e, float((err / tol).max()))
        assert np.linalg.norm(err) <= (rf.half_step("bf16") + 1e-4) * np.linalg.norm(ref), (k13, e)


@pytest.mark.parametrize("kw", [
    dict(), dict(S=40, E=16, n_local=16), dict(S=100, E=1, n_local=1, topk=1), dict(S=30, shared_I=256),
])
def test_experts_of_rows_that_are_not_finite(kw):
    """A token with an infinity or a NaN gives NaN rows; every other row keeps its bits,
    also those of the same expert and the same 16 rows."""
    from moe_decode_layer_router_amd.block import Fp8Block

    cfg = get_config("tiny").with_(**kw)
    blk = Fp8Block(make_fp8_inputs(cfg, 9))
    blk.ids.copy_(torch.arange(cfg.topk)[None] + torch.arange(cfg.S)[:, None]).remainder_(cfg.E)
    blk.bucket()
    blk.expert_ffn()
    clean = blk.y.clone()
    blk.x[2, 5], blk.x[cfg.S - 1, cfg.d - 1] = float("inf"), float("nan")
    blk.expert_ffn()
    torch.cuda.synchronize()
    used, R = int(blk.offsets[-1]), blk.dims.r_max
    token = torch.full((blk.y.shape[0],), -1, device="cuda")
    token[:used] = blk.rows[:used]
    if cfg.shared_I:
        token[R:] = torch.arange(cfg.S, device="cuda")
    bad = (token == 2) | (token == cfg.S - 1)
    assert int(bad.sum()) == 2 * (cfg.topk + bool(cfg.shared_I))
    assert bool(torch.isnan(blk.y[bad]).all()) and torch.equal(blk.y[~bad], clean[~bad])
