"""tests/_fp8_plan.py against the library (no GPU)."""

import random

import pytest

import moe_decode_layer_router_amd as mb
from tests._fp8_plan import gemm_workspace, plan


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_workspace_is_the_plans(out):
    """Its size is that of the plan's tiles and K parts."""
    r = random.Random(3)
    seen = set()
    for _ in range(4000):
        M, N, K = (int(2 ** r.uniform(0, hi)) for hi in (14, 15, 15))
        dims = mb.fp8_dims_from(dict(M=M, N=N, K=K, out_type=mb.MOE_BF16 if out == "bf16" else mb.MOE_FP32))
        assert mb.moe_fp8_gemm_workspace_bytes(dims) == gemm_workspace(M, N, K, out), (M, N, K)
        p = plan(M, N, K, out)
        seen.add((p.form, p.parts > 1))
    want = {(f, s) for f in ("rows", "mid", "tile128") for s in (False, True)}
    assert seen == want | ({("tile256", False)} if out == "bf16" else set())
