// fp8_tile.h -- the FP8 product of many rows, tiled through LDS (device code).
//
// A workgroup of kWN x kWM waves takes 16 kRT kWN weight rows x 16 kTT kWM
// tokens and steps through the 128-K blocks: one block of both operands is
// copied to LDS with direct loads (no registers) while the block before it is
// multiplied, one barrier a block. A wave holds kRT x kTT accumulator tiles; per
// block it multiplies from zero and adds into them with the fp32 factor (token
// scale x weight scale), which costs 4 vector fmas beside each 32-cycle MFMA.
// Weights are copied as packed (a 1 KiB piece is one operand half, read back
// contiguously). Token rows are copied as whole 128-byte lines, the 16-byte
// chunks of row r permuted by chunk ^ (r % 8), so that the reads of 8 rows at
// one chunk fall on different banks.
#pragma once

#include "fp8_dev.h"

namespace moeblk {

typedef const __attribute__((address_space(1))) void* fp8_gptr_t;
typedef __attribute__((address_space(3))) void* fp8_lptr_t;

struct Fp8TileArgs {
  const uint8_t* xq;  // e4m3 rows [M][Kb * 128]
  const float* xs;    // [Kb][M]
  const uint8_t* w;   // packed weight
  const float* ws;    // [Nb][Kb]
  void* out;          // [M][N]
  int M, N, Kb;
  bool out_bf16;
  int tiles_n, tiles_m;
};

// Workgroup b -> tile. Consecutive workgroups go round the 8 XCDs; each XCD
// takes a run of consecutive tiles, ordered in groups of 8 token tiles, so
// that the tiles an XCD works on at one time share operands in its L2.
__device__ __forceinline__ void fp8_tile_of(int b, int tiles_n, int tiles_m, int& tn, int& tm) {
  const int T = tiles_n * tiles_m;
  const int xcd = b & 7, per = T >> 3, rem = T & 7;
  const int t = xcd * per + min(xcd, rem) + (b >> 3);
  const int group = t / (8 * tiles_n);
  const int m0 = group * 8, gm = min(8, tiles_m - m0);
  const int in = t - group * 8 * tiles_n;
  tm = m0 + in % gm;
  tn = in / gm;
}

template <int kRT, int kTT, int kWN, int kWM, bool kExact>
__global__ __launch_bounds__(64 * kWN * kWM) void fp8_tile_kernel(Fp8TileArgs a) {
  constexpr int kWaves = kWN * kWM;
  constexpr int BN = 16 * kRT * kWN, BM = 16 * kTT * kWM;
  constexpr int kWPieces = BN / 8, kXPieces = BM / 8;  // 1 KiB wave loads a block
  static_assert(kWPieces % kWaves == 0 && kXPieces % kWaves == 0, "whole pieces a wave");
  static_assert(kRT * 16 <= 128, "a wave's weight rows share one scale block");
  __shared__ __attribute__((aligned(128))) uint8_t lds[2][(BN + BM) * 128];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int wn = wave % kWN, wm = wave / kWN;
  int tn, tm;
  fp8_tile_of(blockIdx.x, a.tiles_n, a.tiles_m, tn, tm);
  const int Kb = a.Kb, M = a.M;
  const size_t Kp = static_cast<size_t>(Kb) * kFp8Block;

  // this wave's pieces: global addresses at block 0 (rows and row tiles past the
  // end are read as the last ones; their results are not stored)
  const uint8_t* wsrc[kWPieces / kWaves];
  const uint8_t* xsrc[kXPieces / kWaves];
  const int last_rt = fp8_row_tiles(a.N) - 1;
#pragma unroll
  for (int i = 0; i < kWPieces / kWaves; ++i) {
    const int p = wave + i * kWaves;  // piece: row tile p / 2, half p % 2
    const int rt = min(tn * (BN / 16) + (p >> 1), last_rt);
    wsrc[i] = a.w + static_cast<size_t>(rt) * Kb * kFp8TileBytes + (p & 1) * 1024 + lane * 16;
  }
#pragma unroll
  for (int i = 0; i < kXPieces / kWaves; ++i) {
    const int p = wave + i * kWaves;  // piece: rows 8 p .. + 7
    const int row = min(tm * BM + 8 * p + (lane >> 3), M - 1);
    xsrc[i] = a.xq + row * Kp + ((lane & 7) ^ (lane >> 3)) * 16;
  }
  const auto load = [&](int kb, int buf) {
#pragma unroll
    for (int i = 0; i < kWPieces / kWaves; ++i)
      __builtin_amdgcn_global_load_lds((fp8_gptr_t)(wsrc[i] + static_cast<size_t>(kb) * kFp8TileBytes),
                                       (fp8_lptr_t)(&lds[buf][(wave + i * kWaves) * 1024]), 16, 0, 0);
#pragma unroll
    for (int i = 0; i < kXPieces / kWaves; ++i)
      __builtin_amdgcn_global_load_lds((fp8_gptr_t)(xsrc[i] + static_cast<size_t>(kb) * kFp8Block),
                                       (fp8_lptr_t)(&lds[buf][BN * 128 + (wave + i * kWaves) * 1024]),
                                       16, 0, 0);
  };

  int tok[kTT];
  f32x4_t acc[kRT][kTT];
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    tok[t] = min(tm * BM + (wm * kTT + t) * 16 + m16, M - 1);
#pragma unroll
    for (int r = 0; r < kRT; ++r) acc[r][t] = f32x4_t{0, 0, 0, 0};
  }
  const int nb = min((tn * BN + wn * kRT * 16) / 128, (a.N + 127) / 128 - 1);
  const float* wsr = a.ws + static_cast<size_t>(nb) * Kb;
  float xs_next[kTT], ws_next;  // the next block's scales, multiplied once they are needed
  const auto scales = [&](int kb) {
    ws_next = wsr[kb];
#pragma unroll
    for (int t = 0; t < kTT; ++t) xs_next[t] = a.xs[static_cast<size_t>(kb) * M + tok[t]];
  };
  scales(0);
  load(0, 0);
  for (int kb = 0; kb < Kb; ++kb) {
    const int buf = kb & 1;
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's pieces have landed
    float s[kTT];
#pragma unroll
    for (int t = 0; t < kTT; ++t) s[t] = xs_next[t] * ws_next;
    __syncthreads();                     // and everyone's; the other buffer is read out
    if (kb + 1 < Kb) {
      scales(kb + 1);
      load(kb + 1, buf ^ 1);
    }
    const uint8_t* lw = &lds[buf][wn * kRT * kFp8TileBytes + lane * 16];
    const uint8_t* lx = &lds[buf][BN * 128 + (wm * kTT * 16 + m16) * 128];
    const int c0 = ((2 * g) ^ (m16 & 7)) * 16, c1 = ((2 * g + 1) ^ (m16 & 7)) * 16;
    i32x8_t b[kTT];
#pragma unroll
    for (int t = 0; t < kTT; ++t)
      b[t] = join8(*reinterpret_cast<const u32x4_t*>(lx + t * 2048 + c0),
                   *reinterpret_cast<const u32x4_t*>(lx + t * 2048 + c1));
    Bf16Frag be[kExact ? kTT : 1];
    if constexpr (kExact) {
#pragma unroll
      for (int t = 0; t < kTT; ++t) be[t] = e4m3_to_bf16(b[t]);
    }
    // Row tile r's MFMAs are issued while row tile r - 1's results are added: an
    // MFMA's result cannot be read for some 40 cycles, which the additions fill.
    // The scheduling groups keep one MFMA to the 4 additions it hides.
    const auto row_tile = [&](int r) {
      return join8(*reinterpret_cast<const u32x4_t*>(lw + r * kFp8TileBytes),
                   *reinterpret_cast<const u32x4_t*>(lw + r * kFp8TileBytes + 1024));
    };
    i32x8_t w_next = row_tile(0);
    f32x4_t d[kTT];
#pragma unroll
    for (int r = 0; r <= kRT; ++r) {
      const i32x8_t w8 = w_next;
      if (r + 1 < kRT) w_next = row_tile(r + 1);
      Bf16Frag we;
      if constexpr (kExact) we = e4m3_to_bf16(w8);
#pragma unroll
      for (int t = 0; t < kTT; ++t) {
        const f32x4_t old = d[t];
        if (r < kRT) {
          if constexpr (kExact)
            d[t] = mfma_exact_block(we, be[t]);
          else
            d[t] = mfma_fp8_block(w8, b[t]);
        }
        if (r > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[r - 1][t][i] = __builtin_fmaf(old[i], s[t], acc[r - 1][t][i]);
        }
      }
      if constexpr (!kExact) {
        if (r + 1 < kRT) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
          if (r < kRT) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
          if (r > 0) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);    // vector ALU
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // nothing moves into another row tile's step
    }
  }

  // lane: token m16 of a token tile, outputs 4 g .. + 3 of a row tile
  const bool quad = a.N % 4 == 0;
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    const int token = tm * BM + (wm * kTT + t) * 16 + m16;
    if (token >= M) continue;
    const size_t orow = static_cast<size_t>(token) * a.N;
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      const int n0 = tn * BN + (wn * kRT + r) * 16 + 4 * g;
      const f32x4_t v = acc[r][t];
      if (quad) {
        if (n0 < a.N) {
          if (a.out_bf16) {
            const u32x2_t p = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + orow + n0) = p;
          } else {
            *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + orow + n0) = v;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < a.N) {
            if (a.out_bf16)
              static_cast<uint16_t*>(a.out)[orow + n0 + i] =
                  static_cast<uint16_t>(f32_to_bf16_bits(v[i]));
            else
              static_cast<float*>(a.out)[orow + n0 + i] = v[i];
          }
      }
    }
  }
}

}  // namespace moeblk
