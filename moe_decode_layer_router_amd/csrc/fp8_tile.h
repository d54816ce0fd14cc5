// fp8_tile.h -- the FP8 product of many rows, tiled through LDS (device code).
//
// A workgroup of kWN x kWM waves takes 16 kRT kWN weight rows x 16 kTT kWM
// tokens and steps through the 128-K blocks. Both operands are copied to LDS by
// direct loads (no registers). A wave holds kRT x kTT accumulator tiles; a block
// is multiplied from zero and added into them with the fp32 factor (token scale
// x weight scale): 4 vector fmas beside each 32-cycle MFMA (on MI355X 4 fmas an
// MFMA cost 18% over the MFMAs alone, 8 cost 63%).
//
// Step k's work on row tile r, token tile t is one unit: the additions of the
// result d[t] that the row tile before left, then the MFMA that replaces it, so
// an MFMA's latency is covered by the units in between (the last row tile's
// additions fall into the next step). One barrier a step, in front of the last
// row tile but one: each wave has waited for its own copies of step k + 1, so
// behind it all of them have landed, and every wave is done with step k - 1's
// buffers and with step k's token rows (held in registers). The copies of step
// k + 2 start there (weights: 3 buffers, token rows: 2), a full step before they
// are needed, and the first operands of step k + 1 are read during the last row
// tile, so no wave waits for LDS at the start of a step.
//
// 8192 x 4096 x 7168 (256 x 256 tiles): median 231 us, 2.08 PFLOP/s; the fastest of 60
// launches 211. The operand copies alone took 183 us (39 GB/s a CU), so they bound it more
// than the MFMAs do.
//
// Weights are copied as packed (a 1 KiB piece is one operand half, read back
// contiguously). Token rows are copied as whole 128-byte lines, the 16-byte
// chunks of row r permuted by chunk ^ (r % 8), so that the reads of 8 rows at
// one chunk fall on different banks.
#pragma once

#include "fp8_dev.h"

namespace moeblk {

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
  SplitK split;
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
__device__ __forceinline__ void fp8_tile(const Fp8TileArgs& a, uint8_t* lds) {
  constexpr int kWaves = kWN * kWM;
  constexpr int BN = 16 * kRT * kWN, BM = 16 * kTT * kWM;
  constexpr int kWPieces = BN / 8, kXPieces = BM / 8;  // 1 KiB wave loads a block
  static_assert(kWPieces % kWaves == 0 && kXPieces % kWaves == 0, "whole pieces a wave");
  static_assert(kRT * 16 <= 128, "a wave's weight rows share one scale block");
  constexpr int kWBuf = BN * 128, kXBuf = BM * 128;  // LDS bytes of one step's operands
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int wn = wave % kWN, wm = wave / kWN;
  int tn, tm;
  const int tiles = a.tiles_n * a.tiles_m, part = blockIdx.x / tiles;
  fp8_tile_of(blockIdx.x - part * tiles, a.tiles_n, a.tiles_m, tn, tm);
  const int Kb = a.Kb, M = a.M;
  int kb0, kb1;  // this workgroup's K part
  part_range(Kb, a.split.parts, part, kb0, kb1);
  const size_t Kp = static_cast<size_t>(Kb) * kFp8Block;

  // This wave's copies, pieces wave + i kWaves: bases that are the same for the
  // whole wave and 32-bit lane offsets. Rows and row tiles past the end are read
  // as the last ones; their results are not stored.
  const int last_rt = fp8_row_tiles(a.N) - 1;
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  const uint8_t* xbase = a.xq + static_cast<size_t>(tm) * BM * Kp;
  constexpr int kXLoads = kXPieces / kWaves, kLoads = kWPieces / kWaves + kXLoads;
  uint32_t xoff[kXLoads];
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) {
    const int row = min(8 * (uwave + i * kWaves) + (lane >> 3), M - 1 - tm * BM);  // piece: 8 rows
    xoff[i] = static_cast<uint32_t>(row) * static_cast<uint32_t>(Kp) + ((lane & 7) ^ (lane >> 3)) * 16;
  }
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(xbase), 0, static_cast<int>(min(BM, M - tm * BM) * Kp), 0x00020000);
  const int rt0 = tn * (BN / 16), n_rt = min(BN / 16, last_rt + 1 - rt0);
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w) + static_cast<size_t>(rt0) * Kb * kFp8TileBytes, 0,
      static_cast<int>(n_rt * Kb * kFp8TileBytes), 0x00020000);
  // copy i < kLoads of step kb into weight buffer wb, token buffer xb (all offsets are
  // below 2^31)
  const auto copy = [&](int i, int kb, int wb, int xb, uint32_t past = 0) {
    if (i < kXLoads) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xr, (fp8_lptr_t)(lds + 3 * kWBuf + xb * kXBuf + (uwave + i * kWaves) * 1024), 16,
          xoff[i] | past, kb * kFp8Block, 0, 0);
    } else {
      const int p = uwave + (i - kXLoads) * kWaves;  // piece: row tile p / 2, half p % 2
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wr, (fp8_lptr_t)(lds + wb * kWBuf + p * 1024), 16, (lane * 16) | past,
          (min(p >> 1, n_rt - 1) * Kb + kb) * kFp8TileBytes + (p & 1) * 1024, 0, 0);
    }
  };

  // operand reads
  const uint8_t* lw = lds + wn * kRT * kFp8TileBytes + lane * 16;
  const uint8_t* lx = lds + 3 * kWBuf + (wm * kTT * 16 + m16) * 128;
  const int c0 = ((2 * g) ^ (m16 & 7)) * 16, c1 = ((2 * g + 1) ^ (m16 & 7)) * 16;
  const auto read_w = [&](int wb, int r) {
    const uint8_t* p = lw + wb * kWBuf + r * kFp8TileBytes;
    return join8(*reinterpret_cast<const u32x4_t*>(p), *reinterpret_cast<const u32x4_t*>(p + 1024));
  };
  const auto read_x = [&](int xb, int t) {
    const uint8_t* p = lx + xb * kXBuf + t * 2048;
    return join8(*reinterpret_cast<const u32x4_t*>(p + c0), *reinterpret_cast<const u32x4_t*>(p + c1));
  };

  uint32_t tok4[kTT];  // byte offset of the lane's token in a row of scales
  f32x4_t acc[kRT][kTT], d[kTT];
  float s[kTT], s_next[kTT], xs_raw[kTT], ws_raw;
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    tok4[t] = 4u * static_cast<uint32_t>(min(tm * BM + (wm * kTT + t) * 16 + m16, M - 1));
    d[t] = f32x4_t{0, 0, 0, 0};
    s[t] = 0.0f;
#pragma unroll
    for (int r = 0; r < kRT; ++r) acc[r][t] = f32x4_t{0, 0, 0, 0};
  }
  const int nb = min((tn * BN + wn * kRT * 16) / 128, (a.N + 127) / 128 - 1);
  const float* wsr = a.ws + static_cast<size_t>(nb) * Kb;
  const auto load_scales = [&](int kb) {
    ws_raw = wsr[kb];
    const char* xk = reinterpret_cast<const char*>(a.xs + static_cast<size_t>(kb) * M);
#pragma unroll
    for (int t = 0; t < kTT; ++t) xs_raw[t] = *reinterpret_cast<const float*>(xk + tok4[t]);
  };
  const auto wait_all = [&]() {  // every wave's copies have landed, and the scales loaded before
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      asm volatile("" : "+v"(xs_raw[t]));  // used behind the wait, not before it
      s_next[t] = xs_raw[t] * ws_raw;
    }
  };

  load_scales(kb0);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) copy(i, kb0, 0, 0);
  if (kb0 + 1 < kb1) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) copy(i, kb0 + 1, 1, 1);
  }
  wait_all();
  i32x8_t w[2], b[kTT];
  w[0] = read_w(0, 0);
#pragma unroll
  for (int t = 0; t < kTT; ++t) b[t] = read_x(0, t);

  // The steps, one piece of code without branches (several copies of it, or a branch
  // in it, spill the accumulators): the last steps copy, wait and read as if more
  // followed. Their copies get an offset past the buffer's range, which reads
  // nothing; what they leave in LDS is not used.
  int wb = 0;
  for (int kb = kb0; kb < kb1; ++kb) {
    const int xb = (kb - kb0) & 1;
    const int wb1 = wb == 2 ? 0 : wb + 1, wb2 = wb1 == 2 ? 0 : wb1 + 1;
    const uint32_t past = kb + 2 < kb1 ? 0u : 1u << 31;
    float s_now[kTT];
#pragma unroll
    for (int t = 0; t < kTT; ++t) s_now[t] = s_next[t];
    load_scales(min(kb + 1, kb1 - 1));
    Bf16Frag be[kExact ? kTT : 1];
    if constexpr (kExact) {
#pragma unroll
      for (int t = 0; t < kTT; ++t) be[t] = e4m3_to_bf16(b[t]);
    }
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      Bf16Frag we;
      if constexpr (kExact) we = e4m3_to_bf16(w[r & 1]);
      if (r == kRT - 2) wait_all();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < kTT; ++t) {
        f32x4_t& c = acc[r == 0 ? kRT - 1 : r - 1][t];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(d[t][i], s[t], c[i]);
        if (r == 0) s[t] = s_now[t];  // d[t] is this step's from here on
        if constexpr (kExact)
          d[t] = mfma_exact_block(we, be[t]);
        else
          d[t] = mfma_fp8_block(w[r & 1], b[t]);
        if (t == 0 && r + 1 < kRT) w[(r + 1) & 1] = read_w(wb, r + 1);
        if (r == kRT - 1) {  // the next step's first operands
          if (t == 0) w[0] = read_w(wb1, 0);
          b[t] = read_x(xb ^ 1, t);
        }
        {
          constexpr int kUnits = 2 * kTT;  // the last two row tiles
          const int u = (r - (kRT - 2)) * kTT + t;
          if (u >= 0) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
              if (i * kUnits / kLoads == u) copy(i, min(kb + 2, kb1 - 1), wb2, xb, past);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // units stay in order
      }
    }
    wb = wb1;
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // no copy may still be on its way into LDS
#pragma unroll
  for (int t = 0; t < kTT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[kRT - 1][t][i] = __builtin_fmaf(d[t][i], s[t], acc[kRT - 1][t][i]);

  if constexpr (kRT * kTT <= 16) {  // the larger tiles are never split
    f32x4_t(&v)[kRT * kTT] = reinterpret_cast<f32x4_t(&)[kRT * kTT]>(acc);
    if (!join_parts(a.split, tm * a.tiles_n + tn, part, true, v, reinterpret_cast<int*>(lds)))
      return;
  }
  if constexpr (!kExact) {
    // bf16 through LDS (each wave its own part, rows padded by 16 bytes), so that a
    // token's 16 kRT outputs leave as whole lines, 16 bytes a lane
    typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
    constexpr int kPitch = kRT * 32 + 16;
    static_assert(kWaves * 16 * kTT * kPitch <= 3 * kWBuf + 2 * kXBuf, "LDS");
    __syncthreads();  // every wave's operand reads are done
    uint8_t* o = lds + wave * (16 * kTT * kPitch);
#pragma unroll
    for (int t = 0; t < kTT; ++t)
#pragma unroll
      for (int r = 0; r < kRT; ++r) {
        const f32x4_t v = acc[r][t];
        *reinterpret_cast<u32x2_t*>(o + (t * 16 + m16) * kPitch + r * 32 + 8 * g) =
            u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    __syncthreads();
    constexpr int kLanes = 2 * kRT;  // a token
    const int c16 = lane % kLanes;
    const int n0 = tn * BN + wn * 16 * kRT + 8 * c16, left = a.N - n0;
#pragma unroll 4
    for (int i = 0; i < kTT * kRT / 2; ++i) {
      const int row = i * (64 / kLanes) + lane / kLanes, token = tm * BM + wm * 16 * kTT + row;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(o + row * kPitch + 16 * c16);
      if (token >= M) continue;
      uint16_t* to = static_cast<uint16_t*>(a.out) + static_cast<size_t>(token) * a.N + n0;
      if (left >= 8) {
        *reinterpret_cast<u32x4_any_t*>(to) = v;
      } else {
#pragma unroll
        for (int c = 0; c < 7; ++c)
          if (c < left) to[c] = static_cast<uint16_t>(v[c >> 1] >> (16 * (c & 1)));
      }
    }
    return;
  }
  // lane: token m16 of a token tile, outputs 4 g .. + 3 of a row tile
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    const int token = tm * BM + (wm * kTT + t) * 16 + m16;
    const size_t orow = static_cast<size_t>(token) * a.N;
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      const int n0 = tn * BN + (wn * kRT + r) * 16 + 4 * g;
      if (token < M) store4<kExact>(a.out, orow + n0, a.N - n0, acc[r][t], a.out_bf16);
      __builtin_amdgcn_sched_barrier(0);  // one tile's addresses at a time
    }
  }
}

template <int kRT, int kTT, int kWN, int kWM, bool kExact>
__global__ __launch_bounds__(64 * kWN * kWM, kRT * kTT > 32 ? 1 : 2) void fp8_tile_kernel(Fp8TileArgs a) {
  constexpr int kBytes = (3 * 16 * kRT * kWN + 2 * 16 * kTT * kWM) * 128;
  static_assert(kBytes <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(128))) uint8_t lds[kBytes];
  fp8_tile<kRT, kTT, kWN, kWM, kExact>(a, lds);
}

}  // namespace moeblk
