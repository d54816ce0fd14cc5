"""The restated kernel rules of tests/_mx_plan.py: equal to the library's where that can be
seen (workspace sizes), and every kernel and split reached by the sizes of the GPU tests."""

import moe_decode_layer_router_amd as mb
from tests import _mx_plan as mp
from tests import test_gpu_mx as gm
from tests import test_gpu_mx_group as gg


def _sizes(fn):
    return [a for m in fn.pytestmark if m.name == "parametrize" and m.args[0] == "M,N,K" for a in m.args[1]]


def test_workspaces():
    sizes = [1, 15, 16, 17, 32, 33, 63, 64, 65, 100, 129, 256, 300, 512, 1000, 2100, 4097, 20000, 262144]
    for M in sizes:
        for N in (1, 60, 64, 65, 300, 1024, 2049, 4096, 4100, 32768):
            for K in (1, 128, 1000, 1537, 2048, 2305, 3000, 4096, 5000, 8191, 32768):
                d = mb.mx_dims_from(dict(M=M, N=N, K=K))
                assert mb.moe_mx_gemm_workspace_bytes(d) == mp.gemm_workspace(M, N, K), (M, N, K)


def test_products_reach_every_kernel():
    got = {(p.form, p.parts > 1) for p in (mp.plan(*s) for s in gm.SMALL + _sizes(gm.test_product_large_tiles))}
    want = {(f, False) for f in ("rows16", "rows32", "tile64", "tile128", "tile256")}
    assert got == want | {("rows16", True), ("tile64", True)}  # 32 rows a workgroup are never split


def test_experts_reach_every_kernel():
    up = {mp.group_form(T, E, k, n, 2 * I) for T, E, k, n, d, I, _ in gg.CASES + gg.LARGE}  # noqa: E741
    down = {mp.group_form(T, E, k, n, d) for T, E, k, n, d, I, _ in gg.CASES + gg.LARGE}  # noqa: E741
    assert up == down == {"few", "tile64", "tile128", "tile256"}, (up, down)
