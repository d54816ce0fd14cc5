"""What the MXFP4 tiles' copies read (csrc/mx_copy.h, compiled for the host): nothing behind the
readable bytes, whether the hardware's range check counts the scalar offset or not, and every
byte a tile needs."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

import moe_decode_layer_router_amd as mb

CSRC = os.path.join(os.path.dirname(mb.__file__), "csrc")
SRC = """
#define __host__
#define __device__
#include "mx_copy.h"
using namespace moeblk;
static unsigned long long join(MxCopy c) { return (static_cast<unsigned long long>(c.scalar) << 32) | c.lane; }
extern "C" {
unsigned long long x_copy(uint32_t row, int c0, int n, int u) { return join(mx_x_copy(row, c0, n, u)); }
unsigned long long s_copy(uint32_t row, int c0, int n, int v) { return join(mx_s_copy(row, c0, n, v)); }
unsigned long long w_copy(uint32_t lane, int c0, int n, int k, int Kc, int rb, int blocks, int tile, int piece) {
  return join(mx_w_copy(lane, c0, n, k, Kc, rb, blocks, tile, piece));
}
}
"""
TILE = 4352  # bytes of a packed tile


@pytest.fixture(scope="module")
def copies(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx_copy")
    (d / "copy.cpp").write_text(SRC)
    cxx = os.environ.get("CXX", "g++")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "copy.cpp"), "-o", str(d / "copy.so")],
                   check=True)
    L = ctypes.CDLL(str(d / "copy.so"))
    for f in (L.x_copy, L.s_copy, L.w_copy):
        f.restype = ctypes.c_uint64
    return L


def _read(got, size, records):
    """The dwords that a copy of `size` bytes a lane reads: their places from the base, checked
    by the lane offset alone and by the sum with the scalar offset."""
    lane, scalar = got & 0xFFFFFFFF, got >> 32
    at = [lane + 4 * i for i in range(size // 4)]
    alone = [a + scalar for a in at if a < records]
    both = [a + scalar for a in at if a + scalar < records]
    return alone, both


# chunks of a row, and the part of them that a workgroup takes
PARTS = [(kc, 0, kc) for kc in (1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 56, 127, 128, 256)]
PARTS += [(17, 0, 9), (17, 9, 17), (25, 12, 25), (64, 13, 26), (7, 5, 7)]


def _rows(kc):
    """(rows readable, a row's index): the first and the last of a tile, and of what gate_up may read."""
    return [(1, 0), (2, 1), (64, 63), (320, 319), (320, 0), (262144 if kc <= 128 else 320, 262143 if kc <= 128 else 319)]


@pytest.mark.parametrize("Kc,c0,c1", PARTS)
def test_token_copies(copies, Kc, c0, c1):
    n = c1 - c0
    for readable, row in _rows(Kc):
        records = readable * Kc * 64
        assert records <= 1 << 31
        seen = set()
        for u in range((n + 3) // 2 + 1):
            for block in (0, 3, 7):  # 16-byte pieces of a unit's 128
                for read in _read(copies.x_copy(row * Kc * 64 + 16 * block, c0, n, u), 16, records):
                    assert all(0 <= a <= records - 4 for a in read), (u, block)
                    assert not read or 2 * u < n
                    if block in (0, 3) and 2 * u < n:
                        assert read == [row * Kc * 64 + (c0 + 2 * u) * 64 + 16 * block + 4 * i for i in range(4)]
                        seen.add(2 * u)
        assert seen == set(range(0, n, 2))


@pytest.mark.parametrize("Kc,c0,c1", PARTS)
def test_scale_copies(copies, Kc, c0, c1):
    n = c1 - c0
    for readable, row in _rows(Kc):
        records = readable * Kc * 4
        for v in range((n + 8) // 4 + 1):
            for read in _read(copies.s_copy(row * Kc * 4, c0, n, v), 16, records):
                assert all(0 <= a <= records - 4 for a in read), v
                want = {row * Kc * 4 + (c0 + c) * 4 for c in range(4 * v, min(4 * v + 4, n))}
                assert want <= set(read) and (want or not read)
        for read in _read(copies.s_copy(row * Kc * 4, c0, 0, 0), 16, records):  # a copy that reads nothing
            assert not read


@pytest.mark.parametrize("Kc,c0,c1", PARTS)
def test_weight_copies(copies, Kc, c0, c1):
    n = c1 - c0
    for blocks in (1, 3, 4):
        records = blocks * Kc * TILE
        for k in range(n + 4):
            for rb in range(4):
                for lane, size, piece in ((0, 16, 0), (1008, 16, 3072), (0, 4, 4096), (252, 4, 4096)):
                    reads = _read(copies.w_copy(lane, c0, n, k, Kc, rb, blocks, TILE, piece), size, records)
                    for read in reads:
                        at = (min(rb, blocks - 1) * Kc + c0 + k) * TILE + piece + lane
                        assert read == ([at + 4 * i for i in range(size // 4)] if k < n else [])


def test_a_scalar_offset_would_leave_the_buffer():
    """What the checks above are there to see: the last token's last unit of three chunks, with the
    unit in the scalar offset."""
    Kc, rows = 3, 64
    unit = (np.uint64(2 * 64) << np.uint64(32)) | np.uint64((rows - 1) * Kc * 64 + 112)
    alone, _ = _read(int(unit), 16, rows * Kc * 64)
    assert max(alone) >= rows * Kc * 64
