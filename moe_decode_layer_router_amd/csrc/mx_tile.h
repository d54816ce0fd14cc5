// mx_tile.h -- the MXFP4 product of many rows, tiled through LDS (device code).
//
// A workgroup of kWN x kWM waves takes 16 kRT kWN weight rows x 16 kTT kWM rows
// (tokens) and steps through the 128-K chunks; a wave holds kRT x kTT accumulator
// tiles, to which the scaled MFMA adds a chunk's products directly. Both operands and
// their scales are copied to LDS by direct loads (no registers), kStages steps in a
// ring.
//
// Step k's unit (r, t) is one MFMA of row tile r and token tile t. The weight operand of
// row tile r + 1 is read from LDS during row tile r; the tokens' operands stay in
// registers for the step and are replaced by step k + 1's in the last row tile, each
// behind its last use. One barrier a step, in front of the last row tile but one: each
// wave has waited for its own copies of step k + 1, so behind it all of them have
// landed, and every wave is done with step k - 1's buffer. The copies of step
// k + kStages - 1 go there.
//
// Weights are copied as packed (1 KiB pieces, read back contiguously; the scales of a
// row block are a word a lane). Of the tokens a 1 KiB piece is 16 rows' 64 bytes of the
// chunk, the 16-byte blocks of row m permuted by block ^ (m / 2 % 4), so that the reads
// of 8 rows at one block fall on different banks.
#pragma once

#include "mx_dev.h"

namespace moeblk {

typedef __attribute__((address_space(3))) void* mx_lptr_t;

struct MxTile {
  const uint8_t* w;        // the matrix' tiles
  int rb0, row_blocks;     // first row block of this tile, row blocks of the matrix
  const uint8_t *xq, *xs;  // rows that row_of counts from
  uint32_t xq_bytes, xs_bytes;  // readable there
  int Kc, c0, c1;          // chunks of a row; those of this part
};

// vmcnt(n) alone
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n < 64, "6 bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (n & 15) | ((n >> 4) << 14));
}

// row_of(i) gives the row (from p.xq) of the tile's token i, i < 16 kTT kWM
template <int kRT, int kTT, int kWN, int kWM, int kStages, typename F>
__device__ __forceinline__ void mx_tile_body(const MxTile& p, F row_of, uint8_t* lds,
                                             f32x4_t (&acc)[kRT][kTT]) {
  constexpr int kWaves = kWN * kWM;
  constexpr int BN = 16 * kRT * kWN, BM = 16 * kTT * kWM;
  constexpr int kW = BN / 16 / kWaves, kX = BM / 16 / kWaves;  // 1 KiB pieces a wave copies
  constexpr int kSW = (BN / 64 + kWaves - 1) / kWaves, kSX = (BM / 64 + kWaves - 1) / kWaves;
  static_assert(BN / 16 % kWaves == 0 && BM / 16 % kWaves == 0, "whole pieces a wave");
  static_assert(kRT % 4 == 0, "whole row blocks a wave");
  constexpr int kLoads = kW + kX + kSW + kSX;
  constexpr int kXAt = BN * 64, kSWAt = kXAt + BM * 64, kSXAt = kSWAt + BN * 4;
  constexpr int kStage = kSXAt + BM * 4;  // bytes
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int wn = wave % kWN, wm = wave / kWN;
  const int Kc = p.Kc;

  // This wave's copies: bases that are the same for the whole wave and 32-bit lane
  // offsets. Row blocks past the end are read as the last one.
  const int blocks = min(BN / 64, p.row_blocks - p.rb0);
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.w) + static_cast<size_t>(p.rb0) * Kc * kMxTileBytes, 0,
      blocks * Kc * kMxTileBytes, 0x00020000);
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.xq), 0, static_cast<int>(p.xq_bytes), 0x00020000);
  const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.xs), 0, static_cast<int>(p.xs_bytes), 0x00020000);
  uint32_t xoff[kX], soff[kSX];
#pragma unroll
  for (int i = 0; i < kX; ++i) {
    const int m = lane >> 2;
    xoff[i] = static_cast<uint32_t>(row_of(16 * (wave + i * kWaves) + m)) * (Kc * 64u) +
              ((lane & 3) ^ ((m >> 1) & 3)) * 16;
  }
#pragma unroll
  for (int i = 0; i < kSX; ++i)  // with fewer pieces than waves some copy the same ones
    soff[i] = static_cast<uint32_t>(row_of(64 * ((wave + i * kWaves) % (BM / 64)) + lane)) * (Kc * 4u);
  // copy i < kLoads of chunk c into buffer s; `past`: 0, or an offset behind every buffer
  const auto copy = [&](int i, int c, int s, uint32_t past) {
    uint8_t* to = lds + s * kStage;
    if (i < kW) {
      const int q = wave + i * kWaves;  // piece: row tile q
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wr, (mx_lptr_t)(to + q * 1024), 16, (lane * 16) | past,
          (min(q >> 2, blocks - 1) * Kc + c) * kMxTileBytes + (q & 3) * 1024, 0, 0);
    } else if (i < kW + kX) {
      const int q = wave + (i - kW) * kWaves;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (mx_lptr_t)(to + kXAt + q * 1024), 16,
                                               xoff[i - kW] | past, c * 64, 0, 0);
    } else if (i < kW + kX + kSW) {
      const int q = (wave + (i - kW - kX) * kWaves) % (BN / 64);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wr, (mx_lptr_t)(to + kSWAt + q * 256), 4, (lane * 4) | past,
          (min(q, blocks - 1) * Kc + c) * kMxTileBytes + 4096, 0, 0);
    } else {
      const int q = (wave + (i - kW - kX - kSW) * kWaves) % (BM / 64);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (mx_lptr_t)(to + kSXAt + q * 256), 4,
                                               soff[i - kW - kX - kSW] | past, c * 4, 0, 0);
    }
  };

  // operand reads
  const uint8_t* lw = lds + wn * kRT * 1024 + lane * 16;
  const uint8_t* lsw = lds + kSWAt + wn * kRT * 64 + lane * 4;
  const uint8_t* lx = lds + kXAt + wm * kTT * 1024 + m16 * 64 + ((g ^ ((m16 >> 1) & 3)) * 16);
  const uint8_t* lsx = lds + kSXAt + (wm * kTT * 16 + m16) * 4 + g;
  const auto read_w = [&](int s, int r) {
    return *reinterpret_cast<const u32x4_t*>(lw + s * kStage + r * 1024);
  };
  const auto read_sw = [&](int s, int r) {  // of row tiles r .. r + 3
    return *reinterpret_cast<const uint32_t*>(lsw + s * kStage + r * 64);
  };
  const auto read_x = [&](int s, int t) {
    return *reinterpret_cast<const u32x4_t*>(lx + s * kStage + t * 1024);
  };
  const auto read_sx = [&](int s, int t) {
    return static_cast<uint32_t>(lsx[s * kStage + t * 64]);
  };

#pragma unroll
  for (int r = 0; r < kRT; ++r)
#pragma unroll
    for (int t = 0; t < kTT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};

  constexpr uint32_t kPast = 1u << 31;  // behind every buffer: such a copy reads nothing
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int c = p.c0 + s;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) copy(i, min(c, p.c1 - 1), s, c < p.c1 ? 0u : kPast);
  }
  wait_loads<(kStages - 2) * kLoads>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  u32x4_t w[2], x[kTT];
  uint32_t sw[2], sw_next, sx[kTT];
  w[0] = read_w(0, 0);
  sw[0] = read_sw(0, 0);
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    x[t] = read_x(0, t);
    sx[t] = read_sx(0, t);
  }
  int s = 0;
  for (int c = p.c0; c < p.c1; ++c) {
    const int s1 = s + 1 == kStages ? 0 : s + 1, s3 = s == 0 ? kStages - 1 : s - 1;
    const int cn = c + kStages - 1;
    const uint32_t past = cn < p.c1 ? 0u : kPast;
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      if (r == kRT - 2) {  // step c + 1 has landed, step c - 1's buffer is free
        asm volatile("" ::: "memory");
        wait_loads<(kStages - 3) * kLoads>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < kTT; ++t) {
        acc[r][t] = mfma_mx_row(r, w[r & 1], x[t], acc[r][t], sw[(r >> 2) & 1], sx[t]);
        if (t == 0 && r + 1 < kRT) {
          w[(r + 1) & 1] = read_w(s, r + 1);
          if ((r + 1) % 4 == 0) sw[((r + 1) >> 2) & 1] = read_sw(s, r + 1);
        }
        if (r == kRT - 1) {  // the next step's first operands
          x[t] = read_x(s1, t);
          sx[t] = read_sx(s1, t);
          if (t == 0) {
            w[0] = read_w(s1, 0);
            sw_next = read_sw(s1, 0);
          }
        }
        const int u = (r - (kRT - 2)) * kTT + t;  // the copies go along with the last two row tiles
        if (u >= 0) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
            if (i * (2 * kTT) / kLoads == u) copy(i, min(cn, p.c1 - 1), s3, past);
        }
        __builtin_amdgcn_sched_barrier(0);  // units stay in order
      }
    }
    sw[0] = sw_next;
    s = s1;
  }
  wait_loads<0>();  // no copy may still be on its way into LDS
  __syncthreads();  // and every wave's reads are done: the caller may use LDS
}

template <int kRT, int kTT, int kWN, int kWM, int kStages>
constexpr int mx_tile_lds() {
  return kStages * (16 * kRT * kWN + 16 * kTT * kWM) * 68;
}

// Workgroup b of a grid of at least `tiles` -> its tile, or -1: consecutive workgroups
// go round the 8 XCDs, each XCD takes a run of consecutive tiles
__device__ __forceinline__ int mx_xcd_tile(int b, int tiles) {
  const int xcd = b & 7, per = tiles >> 3, rem = tiles & 7;
  const int i = b >> 3;
  if (i >= per + (xcd < rem ? 1 : 0)) return -1;
  return xcd * per + min(xcd, rem) + i;
}
// tile t of tiles_n x tiles_m, in groups of 8 token tiles (kept in one L2)
__device__ __forceinline__ void mx_tile_at(int t, int tiles_n, int tiles_m, int& tn, int& tm) {
  const int group = t / (8 * tiles_n);
  const int m0 = group * 8, gm = min(8, tiles_m - m0);
  const int in = t - group * 8 * tiles_n;
  tm = m0 + in % gm;
  tn = in / gm;
}

// bf16 outputs through LDS (each wave its own part, rows padded by 16 bytes), so that
// they leave as whole lines, 16 bytes a lane: kCols values a token in v(t, m16-row of the
// lane) order; put(t, o) writes the lane's values of token tile t at its row o.
template <int kTT, int kCols, typename Put, typename Row>
__device__ __forceinline__ void mx_store_bf16(uint8_t* lds, Put put, Row row_of, int n_left) {
  typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
  constexpr int kPitch = kCols * 2 + 16, kLanes = kCols / 8;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint8_t* o = lds + wave * (16 * kTT * kPitch);
#pragma unroll
  for (int t = 0; t < kTT; ++t) put(t, o + (t * 16 + (lane & 15)) * kPitch);
  __syncthreads();
  const int c16 = lane % kLanes, left = n_left - 8 * c16;
#pragma unroll 4
  for (int i = 0; i < 16 * kTT * kLanes / 64; ++i) {
    const int row = i * (64 / kLanes) + lane / kLanes;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(o + row * kPitch + 16 * c16);
    uint16_t* to = row_of(row);
    if (!to) continue;
    to += 8 * c16;
    if (left >= 8) {
      *reinterpret_cast<u32x4_any_t*>(to) = v;
    } else {
#pragma unroll
      for (int c = 0; c < 7; ++c)
        if (c < left) to[c] = static_cast<uint16_t>(v[c >> 1] >> (16 * (c & 1)));
    }
  }
}

}  // namespace moeblk
