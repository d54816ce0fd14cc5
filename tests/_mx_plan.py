"""The rules by which the MXFP4 products pick their kernels, restated so that a test can
say which kernel its sizes reach. test_mx_plan_cpu.py holds the first against the library's
workspace sizes."""

from typing import NamedTuple


class Plan(NamedTuple):
    form: str  # rows16, rows32, tile64, tile128, tile256
    tiles: int
    parts: int  # K parts


def _up(a, b):
    return -(-a // b)


def _parts(tiles, kc, least):
    return 1 if tiles > 256 else max(1, min(256 // tiles, kc // least))


def row_tiles(count, bm, over):
    full, rest = divmod(count, bm)
    return full + (rest > (over if full else 0))


def plan(M, N, K) -> Plan:
    kc, tn = _up(K, 128), _up(N, 64)
    form, bm = ("rows16", 16) if M <= 16 or tn * _up(M, 16) <= 256 else ("rows32", 32)
    tiles = tn * _up(M, bm)
    parts = _parts(tiles, kc, 8 if kc >= 32 else 16)
    if M <= 32 or (tiles <= 256 and _up(kc, parts) <= 18):
        return Plan(form, tiles, parts)
    t64 = tn * _up(M, 64)
    if t64 <= 512:
        return Plan("tile64", t64, _parts(t64, kc, 12))
    t128, t256 = _up(N, 128) * _up(M, 128), _up(N, 256) * row_tiles(M, 256, 64)
    if _up(t128, 512) * 66 <= _up(t256, 256) * 100:
        return Plan("tile128", t128, 1)
    return Plan("tile256", t256, 1)


def gemm_workspace(M, N, K) -> int:
    p = plan(M, N, K)
    part = 8192 if p.form.startswith("rows") else 16384
    return 65536 + (p.tiles * p.parts * part if p.parts > 1 else 0)


def group_form(T, E, k, n, N) -> str:
    """Of the experts' products with N weight rows: few, tile64, tile128, tile256."""
    per = T * k // E
    active = min(max(T * k * n // E, 1), n)
    blocks = active * (N // 64)
    if blocks <= 256 and per <= 16:
        return "few"
    if per >= 12 and active * _up(N, 256) * (1 if per < 384 else (per + 128) // 256) >= 200:
        return "tile256"
    return "tile64" if blocks * _up(per, 64) <= 512 else "tile128"
