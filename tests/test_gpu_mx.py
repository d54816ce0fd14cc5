"""GPU parity of the MXFP4 calls for many rows against the 64-bit references of
tests/_ref_many.py (which derives the tolerances): moe_mx_quant and moe_mx_dequant bit
for bit, the products within the bound of an fp32 accumulation plus one rounding."""

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


def _rows(M, K, kind, seed):
    r = np.random.default_rng([seed, M, K])
    x = r.standard_normal((M, K)) * np.exp(r.standard_normal((M, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(TT[kind])


def _guarded(shape, dtype, fill=0xA5):
    """A tensor inside a larger buffer whose bytes behind it hold `fill`."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n + 4096,), fill, dtype=torch.uint8, device="cuda")
    return raw[:n].view(dtype).view(shape), raw[n:]


def _intact(*guards):
    torch.cuda.synchronize()
    assert all(bool((g == 0xA5).all()) for g in guards), "wrote behind its outputs"


def _quant(x, dims):
    kc = -(-dims.K // 128)
    q, g1 = _guarded((dims.M, kc * 64), torch.uint8)
    s, g2 = _guarded((dims.M, kc * 4), torch.uint8)
    mb.moe_mx_quant(dims, x, q, s)
    _intact(g1, g2)
    return q, s


def _held(v):
    """What bf16 and fp32 hold of MXFP4 values: all but those of 2^128 and more (4 x 2^126, which
    the largest numbers round to)."""
    return np.where(np.abs(v) >= 2.0**128, np.sign(v) * np.inf, v)


def _check_quant(x, kind):
    M, K = x.shape
    dims = mb.mx_dims_from(dict(M=M, K=K, in_type=KIND[kind]))
    q, s = _quant(x.cuda(), dims)
    code, sr = rm.mx_quant(x.double().numpy())
    assert np.array_equal(to_np(s), sr)
    got = rm.mx_unpack(to_np(q))
    # the sign of a zero is kept or not
    assert np.array_equal(np.where(got == 8, 0, got), np.where(code == 8, 0, code))
    for back in ("bf16", "fp32"):
        bd = mb.mx_dims_from(dict(M=M, K=K, out_type=KIND[back]))
        v, g = _guarded((M, K), TT[back])
        mb.moe_mx_dequant(bd, q, s, v)
        _intact(g)
        assert np.array_equal(v.double().cpu().numpy(), _held(rm.mx_values(code, sr)[:, :K]), equal_nan=True)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 32), (1, 128), (2, 31), (2, 33), (3, 129), (16, 1000), (5, 130), (77, 2120),
                                 (300, 4096), (1, 32768), (2000, 36), (7, 127)])
def test_quant_and_back(M, K, kind):
    _check_quant(_rows(M, K, kind, 0), kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_quant_edge_values(kind):
    x = _rows(24, 300, kind, 1)
    big = torch.finfo(TT[kind]).max
    x[0] = 0
    x[1] = 1e-39  # subnormal
    x[2, :140] = 7.0
    x[3, :40] = 6.96875  # below 7: rounds to 6
    x[4] = big
    x[5, 7] = -big
    x[6, 5] = float("inf")
    x[7, 200] = float("nan")
    x[8, 299] = float("-inf")
    x[9] = 2.0**-127
    x[10, ::3] = 2.0**-130
    x[11] = -0.0
    x[12, :32] = torch.linspace(0, 6, 32)
    x[13, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])  # ties
    x[14, :8] = -x[13, :8]
    x[15, :64] = torch.tensor([2.0**-126, 2.0**-125 * 1.75] * 32)
    x[16, 0] = 2.0**127
    x[17, 31] = 1e-45 if kind == "fp32" else 2.0**-133
    _check_quant(x, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_quant_every_binade(kind):
    """Magnitudes over the type's whole range, and mantissas on both sides of 7."""
    m = torch.tensor([1.0, 1.25, 1.5, 1.7421875, 1.75, 1.7578125, 1.9921875])
    e = torch.arange(-133, 128, dtype=torch.float64)
    v = (m[:, None].double() * torch.exp2(e)[None, :]).float().to(TT[kind])
    x = torch.zeros((v.numel(), 32), dtype=TT[kind])
    x[:, 3] = v.reshape(-1)
    x[:, 9] = (-v.float() * 0.4375).to(TT[kind]).reshape(-1)
    _check_quant(x, kind)


@pytest.mark.parametrize("back", ["bf16", "fp32"])
def test_dequant_every_code_and_scale(back):
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 8))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    dims = mb.mx_dims_from(dict(M=256, K=128, out_type=KIND[back]))
    v = torch.empty((256, 128), dtype=TT[back], device="cuda")
    mb.moe_mx_dequant(dims, torch.from_numpy(rm.mx_pack(code)).cuda(), torch.from_numpy(s).cuda(), v)
    assert np.array_equal(v.double().cpu().numpy(), _held(rm.mx_values(code, s)), equal_nan=True)


# ------------------------------------------------------------------ products


def _weight(N, K, seed, lo=115, hi=122):
    """Canonical bytes [N, Kp / 2], [N, Kp / 32], the columns past K holding anything, and the values."""
    r = np.random.default_rng([seed, N, K])
    code = r.integers(0, 16, (N, rm.padded(K))).astype(np.uint8)
    s = r.integers(lo, hi, (N, rm.padded(K) // 32)).astype(np.uint8)
    full = -(-K // 32)
    s[:, full:] = 255
    return rm.mx_pack(code), s, rm.mx_values(code[:, :32 * full], s[:, :full])[:, :K]


def _run_gemm(dims, xq, xs, x, q, s, ws=None):
    """Both calls: the outputs have to be the same bits."""
    packed, g0 = _guarded((mb.moe_packed_mx_bytes(dims),), torch.uint8)
    mb.moe_pack_mx(dims, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    out_t = torch.bfloat16 if dims.out_type == mb.MOE_BF16 else torch.float32
    out, g1 = _guarded((dims.M, dims.N), out_t)
    if ws is None:
        ws = torch.zeros(mb.moe_mx_proj_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_mx_gemm(dims, xq, xs, packed, out, ws)
    _intact(g0, g1)
    out2, g2 = _guarded((dims.M, dims.N), out_t)
    mb.moe_mx_proj(dims, x, packed, out2, ws)
    _intact(g2)
    assert torch.equal(out.view(torch.uint8), out2.view(torch.uint8))
    return out


def _check_product(M, N, K, kind, out, seed=0, x=None):
    dims = mb.mx_dims_from(dict(M=M, N=N, K=K, in_type=KIND[kind], out_type=KIND[out]))
    x = _rows(M, K, kind, seed) if x is None else x
    q, s, w = _weight(N, K, seed)
    xq, xs = _quant(x.cuda(), dims)
    got = _run_gemm(dims, xq, xs, x.cuda(), q, s).double().cpu().numpy()
    code, sx = rm.mx_quant(x.double().numpy())
    ref, mag = rm.product(rm.mx_values(code, sx)[:, :K], w)
    tol = rm.product_tol(mag, K) + rm.half_step(out) * np.abs(ref)
    bad = np.abs(got - ref) > tol * 1.0001
    assert not bad.any(), (np.argwhere(bad)[:5], float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


SMALL = [(1, 1, 1), (1, 16, 128), (1, 64, 4096), (2, 17, 129), (16, 100, 300), (15, 8200, 256), (16, 65, 2048), (1, 7, 32768),
         (17, 64, 128), (32, 33, 500), (31, 4100, 130), (33, 64, 1000), (64, 129, 384), (63, 4099, 256), (64, 16, 4096),
         (65, 100, 200), (77, 4099, 2120), (100, 1, 77), (129, 500, 640), (200, 4100, 1500), (300, 4096, 1024), (1000, 1000, 1000),
         (5, 300, 4100), (16, 4096, 1030), (24, 700, 8191), (32, 128, 3999), (33, 100, 5000), (64, 1024, 3080), (100, 64, 20000),
         (512, 4096, 128), (520, 4096, 300), (2100, 2048, 257), (1000, 64, 4096), (2048, 60, 700), (333, 500, 2304), (8000, 17, 33),
         (129, 2000, 3000), (900, 900, 2500)]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", SMALL)
def test_product(M, N, K, out):
    _check_product(M, N, K, "bf16", out)


@pytest.mark.parametrize("M,N,K", [(1, 40, 77), (5, 1000, 3000), (16, 4096, 512), (40, 130, 300), (300, 300, 300)])
def test_product_of_fp32_rows(M, N, K):
    _check_product(M, N, K, "fp32", "bf16")
    _check_product(M, N, K, "fp32", "fp32")


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 384), (4097, 4099, 130), (4500, 4096, 1), (5000, 4200, 640), (256, 65536 // 2, 128),
                                   (2048, 2048, 1100)])
def test_product_large_tiles(M, N, K, out):
    _check_product(M, N, K, "bf16", out)


@pytest.mark.parametrize("M,N,K", [(3, 200, 512), (30, 200, 512), (64, 300, 1024), (200, 4200, 640), (5000, 4200, 256)])
def test_product_exact_where_sums_fit(M, N, K):
    """Scales of 1: all sums are multiples of 1/4 below 2^22 and come out exact, whatever the
    order, a cancelling pair of the largest products included."""
    r = np.random.default_rng([M, N])
    code = r.integers(0, 16, (M, K)).astype(np.uint8)
    wcode = r.integers(0, 16, (N, K)).astype(np.uint8)
    code[:, 0], code[:, K - 1] = 7, 15
    wcode[:, 0], wcode[:, K - 1] = 7, 7
    one = lambda n: np.full((n, K // 32), 127, np.uint8)  # noqa: E731
    dims = mb.mx_dims_from(dict(M=M, N=N, K=K, in_type=mb.MOE_FP32, out_type=mb.MOE_FP32))
    xv = rm.mx_values(code, one(M))
    got = _run_exact(dims, code, one(M), wcode, one(N))
    assert np.array_equal(got, xv @ rm.mx_values(wcode, one(N)).T)


def _run_exact(dims, code, sx, wcode, sw):
    packed = torch.empty(mb.moe_packed_mx_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_pack_mx(dims, torch.from_numpy(rm.mx_pack(wcode)).cuda(), torch.from_numpy(sw).cuda(), packed)
    out = torch.empty((dims.M, dims.N), device="cuda")
    ws = torch.zeros(mb.moe_mx_gemm_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mb.moe_mx_gemm(dims, torch.from_numpy(rm.mx_pack(code)).cuda(), torch.from_numpy(sx).cuda(), packed, out, ws)
    return out.double().cpu().numpy()


@pytest.mark.parametrize("M,N,K", [(4, 100, 512), (40, 100, 512), (300, 300, 512), (5000, 4200, 256)])
def test_product_of_any_scales(M, N, K):
    """Scale bytes of either side over the whole range whose sums stay in fp32's, NaN scales."""
    r = np.random.default_rng([M, N, 2])
    code = r.integers(0, 16, (M, K)).astype(np.uint8)
    wcode = r.integers(0, 16, (N, K)).astype(np.uint8)
    sx = r.integers(40, 170, (M, K // 32)).astype(np.uint8)
    sw = r.integers(90, 200, (N, K // 32)).astype(np.uint8)
    sx[1, 2] = 255
    sw[7, 1] = 255
    dims = mb.mx_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32))
    got = _run_exact(dims, code, sx, wcode, sw)
    xv, wv = rm.mx_values(code, sx), rm.mx_values(wcode, sw)
    nan = np.isnan(xv).any(axis=1)[:, None] | np.isnan(wv).any(axis=1)[None, :]
    assert np.array_equal(np.isnan(got), nan)
    ref, mag = rm.product(np.nan_to_num(xv), np.nan_to_num(wv))
    assert (np.abs(got - ref) <= rm.product_tol(mag, K) + rm.U24 * np.abs(ref))[~nan].all()


def test_rows_that_are_not_finite_stay_alone():
    for M in (3, 40, 200):
        x = _rows(M, 700, "bf16", 3)
        x[1, 5] = float("inf")
        x[2, 600] = float("nan")
        dims = mb.mx_dims_from(dict(M=M, N=200, K=700, out_type=mb.MOE_FP32))
        q, s, w = _weight(200, 700, 3)
        xq, xs = _quant(x.cuda(), dims)
        got = _run_gemm(dims, xq, xs, x.cuda(), q, s)
        nan = torch.isnan(got).any(dim=1)
        assert nan[1] and nan[2] and int(nan.sum()) == 2 and bool(torch.isnan(got[1:3]).all())


def test_gemm_workspace_is_left_ready():
    """One workspace over products of several sizes, split over K and not, in turn."""
    sizes = [(1, 512, 8192), (64, 256, 8192), (300, 500, 4096), (8, 1024, 4096), (1, 512, 8192)]
    all_dims = [mb.mx_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32)) for M, N, K in sizes]
    ws = torch.zeros(max(mb.moe_mx_proj_workspace_bytes(d) for d in all_dims), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for d in all_dims:
            x = _rows(d.M, d.K, "bf16", 4)
            q, s, w = _weight(d.N, d.K, 4)
            xq, xs = _quant(x.cuda(), d)
            a = _run_gemm(d, xq, xs, x.cuda(), q, s, ws)
            b = _run_gemm(d, xq, xs, x.cuda(), q, s)
            assert torch.equal(a, b)


def test_products_in_graphs_that_share_a_workspace():
    """Two captured products of one workspace, replayed in turn on new rows, eager calls on the
    same workspace between; split over K and not, quantised in the kernel and in front of it."""
    sizes = [(1, 512, 8192), (64, 256, 8192), (300, 500, 4096), (300, 4096, 1024), (40, 130, 300)]
    dims = [mb.mx_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32)) for M, N, K in sizes]
    ws = torch.zeros(max(mb.moe_mx_proj_workspace_bytes(d) for d in dims), dtype=torch.uint8, device="cuda")
    calls = []
    for d in dims:
        q, s, _ = _weight(d.N, d.K, 4)
        packed = torch.empty(mb.moe_packed_mx_bytes(d), dtype=torch.uint8, device="cuda")
        mb.moe_pack_mx(d, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
        x = _rows(d.M, d.K, "bf16", 4).cuda()
        calls.append((d, x, packed, torch.empty((d.M, d.N), device="cuda"), ws))
    stream = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            mb.moe_mx_proj(*c)
        graphs.append(g)
    for i in range(3):
        for c in calls:
            c[1].copy_(_rows(c[0].M, c[0].K, "bf16", 10 + i))
        want = []
        for c in calls:
            mb.moe_mx_proj(*c)
            want.append(c[3].clone())
            c[3].zero_()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c[3], w) for c, w in zip(calls, want)), i


def test_products_on_two_streams():
    """Calls at once, each with its own workspace."""
    M, N, K = 16, 1024, 8192
    d = mb.mx_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_FP32))
    q, s, _ = _weight(N, K, 6)
    packed = torch.empty(mb.moe_packed_mx_bytes(d), dtype=torch.uint8, device="cuda")
    mb.moe_pack_mx(d, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), packed)
    xs = [_rows(M, K, "bf16", i).cuda() for i in range(2)]
    ws = [torch.zeros(mb.moe_mx_proj_workspace_bytes(d), dtype=torch.uint8, device="cuda") for _ in xs]
    want = []
    for x, w in zip(xs, ws):
        out = torch.empty((M, N), device="cuda")
        mb.moe_mx_proj(d, x, packed, out, w)
        want.append(out)
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[torch.zeros((M, N), device="cuda") for _ in range(20)] for _ in xs]
    torch.cuda.synchronize()
    for i in range(20):
        for x, w, o, st in zip(xs, ws, outs, streams):
            mb.moe_mx_proj(d, x, packed, o[i], w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for w, many in zip(want, outs) for o in many)


def test_quant_behind_2_to_32_bytes():
    M, K = 262144, 16384
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(9))
    dims = mb.mx_dims_from(dict(M=M, K=K))
    q = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((M, K // 32), dtype=torch.uint8, device="cuda")
    mb.moe_mx_quant(dims, x, q, s)
    code, sr = rm.mx_quant(x[-5:].double().cpu().numpy())
    assert np.array_equal(to_np(s[-5:]), sr)
    got = rm.mx_unpack(to_np(q[-5:]))
    assert np.array_equal(np.where(got == 8, 0, got), np.where(code == 8, 0, code))
    back = torch.empty_like(x)
    mb.moe_mx_dequant(dims, q, s, back)
    assert np.array_equal(back[-5:].double().cpu().numpy(), rm.mx_values(code, sr))
