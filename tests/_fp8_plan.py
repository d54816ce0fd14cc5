"""The rule by which a product of rows and an FP8 weight picks its kernel, restated
so that a test can say which kernel its sizes reach. test_fp8_plan_cpu.py holds it
against the library's workspace sizes."""

from typing import NamedTuple


class Plan(NamedTuple):
    form: str  # rows, mid, tile128, tile256
    tiles: int
    parts: int  # K parts
    exact: bool  # block sums in fp32 (else the e4m3 matrix instruction's)


def _up(a, b):
    return -(-a // b)


def _parts(tiles, kb, least):
    return 1 if tiles > 256 else max(1, min(256 // tiles, kb // least))


def plan(M, N, K, out) -> Plan:
    kb = _up(K, 128)
    if M <= 16:
        tiles = _up(N, 16 if N <= 8192 else 64)
        return Plan("rows", tiles, _parts(tiles, kb, 16), True)
    mid = M <= 64 or _up(N, 64) * _up(M, 64) <= 320
    exact = out == "fp32" or (M <= 128 and mid)
    if mid:
        groups = _up(M, 32 if M <= 32 else 64)
        tiles = groups * (_up(N, 32) if _up(N, 32) * groups <= 256 else _up(N, 64))
        return Plan("mid", tiles, _parts(tiles, kb, 8), exact)
    t256, t128 = _up(N, 256) * _up(M, 256), _up(N, 128) * _up(M, 128)
    if out == "bf16" and _up(t256, 256) * 190 <= _up(t128, 512) * 125:
        return Plan("tile256", t256, 1, exact)
    return Plan("tile128", t128, _parts(t128, kb, 8), exact)


def gemm_workspace(M, N, K, out) -> int:
    p = plan(M, N, K, out)
    part = {"rows": 16384, "mid": 16384, "tile128": 65536, "tile256": 65536}[p.form]
    return 65536 + (p.tiles * p.parts * part if p.parts > 1 else 0)
