// mx_tile.h -- the MXFP4 product of many rows, tiled through LDS (device code).
//
// A workgroup of kWN x kWM waves takes 64 kWN weight rows x 32 kT kWM rows
// (tokens) and steps through the 128-K chunks; a wave holds 2 x kT accumulators of
// 32 x 32, to which the 32x32x64 scaled MFMA adds half a chunk's products directly (alone,
// with one wave a SIMD, it reached 6.4 PFLOP/s on random codes, the 16x16x128 one 4.5).
//
// Both operands and their scales are copied to LDS by direct loads (no registers). What a
// copy costs is the cache lines it touches, about 3.7 cycles each, whole or not (8192 x
// 4096 x 7168 on 256 x 256 tiles, copies alone: 101 us with the tokens' scales fetched
// chunk by chunk, 64 lines a load, and 64 bytes of a token row at a time; 69 without the
// scales). So weights come as packed, 1 KiB pieces of 8 lines, in a ring of kWRing chunks;
// token rows by whole lines, two chunks at once, and their scales four chunks at once, in
// rings of two.
//
// A step is one chunk: 4 units of kT MFMAs, unit (h, q) being half h of the chunk and
// 32 weight rows. Its weight operand is read from LDS two units ahead; the tokens'
// operands of a step stay in registers, replaced by the next step's in the last two units.
// One barrier a step, in front of those: each wave has waited for its own copies of step
// k + 1, so behind it all of them have landed, and every wave is done with step k - 1's
// weights and holds step k's tokens. The copies that replace those (a batch) go out from
// there to the next barrier, one to two steps before they are needed.
//
// Lane (row or token l % 32, MX block l / 32 of the half). The 16-byte blocks of token
// row m are permuted by block ^ (m / 2 % 8), so that the reads of 16 rows at one block fall
// on different banks. Of a weight row block's scale words (a byte a row tile of 16) the
// lane's own two bytes are shifted to places 0 and 2; so are those of a token's word (a byte a
// block).
#pragma once

#include <type_traits>

#include "mx_copy.h"
#include "mx_dev.h"

namespace moeblk {

typedef __attribute__((address_space(3))) void* mx_lptr_t;
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kQ = 2;  // units of 32 weight rows a wave: a row block
constexpr int kWRing = 4, kXRing = 2;

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

// D[32x32] += A[32x64] B[64x32]: scales from byte kA of sa, byte kB of sb. D: lane's
// column l % 32, element i in row 8 (i / 4) + 4 (l / 32) + i % 4.
template <int kA, int kB>
__device__ __forceinline__ f32x16_t mfma_mx32(u32x4_t a, u32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, kA, (int)sa, kB, (int)sb);
}

// q, h: compile-time after unrolling
__device__ __forceinline__ f32x16_t mfma_mx32_at(int q, int h, u32x4_t a, u32x4_t b, f32x16_t c,
                                                 uint32_t sa, uint32_t sb) {
  if (q & 1) return h ? mfma_mx32<2, 2>(a, b, c, sa, sb) : mfma_mx32<2, 0>(a, b, c, sa, sb);
  return h ? mfma_mx32<0, 2>(a, b, c, sa, sb) : mfma_mx32<0, 0>(a, b, c, sa, sb);
}

template <int kT, int kWN, int kWM>
struct MxTileShape {
  static constexpr int kWaves = kWN * kWM;
  static constexpr int BN = 32 * kQ * kWN, BM = 32 * kT * kWM;
  static constexpr int kWBuf = BN * 68, kXBuf = BM * 128, kSBuf = BM * 16;  // bytes
  static constexpr int kXAt = kWRing * kWBuf, kSAt = kXAt + kXRing * kXBuf;
  static constexpr int kLds = kSAt + kXRing * kSBuf + 1024;
  static_assert(BN / 16 % kWaves == 0 && BM / 8 % kWaves == 0, "whole pieces a wave");
  static_assert(kLds <= 160 * 1024, "LDS");
  // what the outputs pass through behind the last step
  static_assert(kWaves * 32 * (32 * kQ * 4 + 16) <= kLds && kWaves * 32 * kT * 16 <= kLds, "LDS");
};

// row_of(i) gives the row (from p.xq) of the tile's token i
template <int kT, int kWN, int kWM, typename F>
__device__ __forceinline__ void mx_tile_body(const MxTile& p, F row_of, uint8_t* lds,
                                             f32x16_t (&acc)[kQ][kT]) {
  using S = MxTileShape<kT, kWN, kWM>;
  constexpr int kWaves = S::kWaves, BN = S::BN, BM = S::BM;
  constexpr int kW = BN / 16 / kWaves, kX = BM / 8 / kWaves;  // 1 KiB pieces a wave copies
  constexpr int kSW = (BN / 64 + kWaves - 1) / kWaves, kSX = (BM / 64 + kWaves - 1) / kWaves;
  constexpr int kUnits = 2 * kQ;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int m32 = lane & 31, hi = lane >> 5;
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
  for (int i = 0; i < kX; ++i) {  // a piece: 8 rows' 128 bytes
    const int m = lane >> 3;
    xoff[i] = static_cast<uint32_t>(row_of(8 * (wave + i * kWaves) + m)) * (Kc * 64u) +
              ((lane & 7) ^ (4 * ((wave + i * kWaves) & 1) + (m >> 1))) * 16;
  }
#pragma unroll
  for (int i = 0; i < kSX; ++i)
    soff[i] = static_cast<uint32_t>(row_of(64 * min(wave + i * kWaves, BM / 64 - 1) + lane)) * (Kc * 4u);
  // Copies of weight chunk k, of token unit u (chunks 2 u, 2 u + 1), of scale unit v (chunks
  // 4 v .. 4 v + 3), all counted from p.c0; behind the last chunk they read nothing (an offset
  // behind every buffer) or what is not used (mx_copy.h).
  const int n = p.c1 - p.c0;
  const auto copy_w = [&](int i, int k) {
    uint8_t* to = lds + (k & (kWRing - 1)) * S::kWBuf;
    if (i < kW) {
      const int q = wave + i * kWaves;  // piece: row tile of 16
      const MxCopy at = mx_w_copy(lane * 16, p.c0, n, k, Kc, q >> 2, blocks, kMxTileBytes, (q & 3) * 1024);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (mx_lptr_t)(to + q * 1024), 16, at.lane, at.scalar, 0, 0);
    } else {
      const int q = (wave + (i - kW) * kWaves) % (BN / 64);
      const MxCopy at = mx_w_copy(lane * 4, p.c0, n, k, Kc, q, blocks, kMxTileBytes, 4096);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (mx_lptr_t)(to + BN * 64 + q * 256), 4, at.lane, at.scalar, 0, 0);
    }
  };
  const auto copy_x = [&](int i, int u) {
    const MxCopy at = mx_x_copy(xoff[i], p.c0, n, u);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        xr, (mx_lptr_t)(lds + S::kXAt + (u & 1) * S::kXBuf + (wave + i * kWaves) * 1024), 16, at.lane, at.scalar, 0, 0);
  };
  const auto copy_s = [&](int i, int v, bool real = true) {  // !real: reads nothing
    const int q = wave + i * kWaves;
    real = real && q < BM / 64;  // with fewer pieces than waves some have none
    const MxCopy at = mx_s_copy(soff[i], p.c0, real ? n : 0, v);
    const int to = real ? (v & 1) * S::kSBuf + q * 1024 : kXRing * S::kSBuf;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (mx_lptr_t)(lds + S::kSAt + to), 16, at.lane, at.scalar, 0, 0);
  };

  // operand reads of step k
  const int wl = (m32 >> 4) * 1024 + (hi * 16 + (m32 & 15)) * 16;
  const uint8_t* lw = lds + wn * kQ * 2048 + wl;
  const uint8_t* lsw = lds + BN * 64 + wn * kQ * 128 + (hi * 16 + (m32 & 15)) * 4;
  const int swsh = (m32 >> 4) * 8;
  const auto read_w = [&](int k, int unit) {  // half unit / kQ, 32 rows unit % kQ
    return *reinterpret_cast<const u32x4_t*>(lw + (k & (kWRing - 1)) * S::kWBuf + unit % kQ * 2048 +
                                             unit / kQ * 512);
  };
  const auto read_sw = [&](int k, int unit) {  // of units unit, unit + 1: a row block
    return *reinterpret_cast<const uint32_t*>(lsw + (k & (kWRing - 1)) * S::kWBuf + unit % kQ * 128 +
                                              unit / kQ * 128);
  };
  const int row = wm * kT * 32 + m32;
  const uint8_t* lx = lds + S::kXAt + row * 128;
  const uint8_t* lsx = lds + S::kSAt + row * 16;
  const auto read_x = [&](int k, int h, int t) {
    const int block = 4 * (k & 1) + 2 * h + hi;
    return *reinterpret_cast<const u32x4_t*>(lx + ((k >> 1) & 1) * S::kXBuf + t * 4096 +
                                             (block ^ ((row >> 1) & 7)) * 16);
  };
  const auto read_sx = [&](int k, int t) {  // of chunks k, k + 1 (k even): a word each
    return *reinterpret_cast<const u32x2_t*>(lsx + ((k >> 2) & 1) * S::kSBuf + t * 512 + (k & 2) * 4);
  };

#pragma unroll
  for (int q = 0; q < kQ; ++q)
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[q][t][i] = 0.0f;

  // Order of the copies, oldest first: what the first step needs, then what each
  // barrier's batch brings: at step k's weights k + 3, at odd steps token unit (k + 3) / 2,
  // at every fourth (k % 4 = 3) scale unit (k + 5) / 4, and a copy that reads nothing at the
  // odd ones between, so that the steps are one piece of code without branches (which the
  // compiler would move MFMAs across). The two batches in front of step 0 are those of steps
  // -2 and -1.
#pragma unroll
  for (int i = 0; i < kSX; ++i) copy_s(i, 0);
#pragma unroll
  for (int i = 0; i < kX; ++i) copy_x(i, 0);
#pragma unroll
  for (int i = 0; i < kW + kSW; ++i) copy_w(i, 0);
  // Loads of a batch (an odd step's has the tokens' ones, in front). They go along with the
  // kSlots MFMAs up to the next barrier: all at once, right behind a barrier, they queue and
  // hold up the waves that issue them (8192 x 4096 x 7168: 119.6 us, spread 115.5).
  constexpr int kEven = kW + kSW, kOddLoads = kX + kSX + kEven;
  constexpr int kSlots = kUnits * kT;
  const auto batch = [&](int k, auto odd, int slot) {
    constexpr bool kOdd = decltype(odd)::value;
    constexpr int kN = kOdd ? kOddLoads : kEven;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (i * kSlots / kN != slot) continue;
      const int j = kOdd ? i - kX - kSX : i;
      if (j >= 0)
        copy_w(j, k + 3);
      else if (i < kSX)
        copy_s(i, (k + 5) >> 2, (k & 3) == 3);
      else
        copy_x(i - kSX, (k + 3) >> 1);
    }
  };
  const std::true_type odd_step;
  const std::false_type even_step;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) batch(-2, even_step, i);
  // the rest of batch -1 goes along with step 0, like any other's with the step behind it
  constexpr int kHead = 2 * kT;  // slots in front of the step's end
  constexpr int kHeadLoads = (kHead * kOddLoads + kSlots - 1) / kSlots;
#pragma unroll
  for (int i = 0; i < kHead; ++i) batch(-1, odd_step, i);
  wait_loads<kEven + kHeadLoads>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  u32x4_t w[4], x[2][kT];
  uint32_t sw = 0, sw_raw, sx[kT];
  u32x2_t sx_raw[kT];
  w[0] = read_w(0, 0);
  w[1] = read_w(0, 1);
  sw_raw = read_sw(0, 0);
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    x[0][t] = read_x(0, 0, t);
    x[1][t] = read_x(0, 1, t);
    sx_raw[t] = read_sx(0, t);
  }

  // one step; kOdd: k is odd
  const auto step = [&](int k, auto odd) {
    constexpr bool kOdd = decltype(odd)::value;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (u == kUnits - 2) {
        // all but the batch of step k - 1 have landed: that is weights, tokens and scales of
        // step k + 1
        asm volatile("" ::: "memory");
        // the step's second tokens are not in use yet: wait for them, since others may replace
        // them behind the barrier
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
        wait_loads<kOdd ? kEven : kOddLoads>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      constexpr int kLast = kUnits - 1;
      // operands two units ahead
      const int un = u + 2 < kUnits ? u + 2 : u + 2 - kUnits;
      const int kn = u + 2 < kUnits ? k : k + 1;
      if ((u & 1) == 0) sw = sw_raw >> swsh;
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        if (u == 0) sx[t] = sx_raw[t][kOdd] >> (8 * hi);
        acc[u % kQ][t] = mfma_mx32_at(u, u / kQ, w[u & 3], x[u / kQ][t], acc[u % kQ][t], sw, sx[t]);
        if (t == 0) {
          w[(u + 2) & 3] = read_w(kn, un);
          if ((u & 1) == 0) sw_raw = read_sw(kn, un);
        }
        if (u == kLast - 1) {
          x[0][t] = read_x(k + 1, 0, t);
          if constexpr (kOdd) sx_raw[t] = read_sx(k + 1, t);
        }
        if (u == kLast) {
          x[1][t] = read_x(k + 1, 1, t);
        }
        // copies: of this step's batch behind its barrier, of the last one's before
        if (u >= kLast - 1)
          batch(k, odd, (u - (kLast - 1)) * kT + t);
        else
          batch(k - 1, std::integral_constant<bool, !kOdd>(), (u + 2) * kT + t);
      }
    }
  };
  int k = 0;
  for (; k + 1 < n; k += 2) {
    step(k, std::false_type());
    step(k + 1, std::true_type());
  }
  if (k < n) step(k, std::false_type());
  wait_loads<0>();  // no copy may still be on its way into LDS
  __syncthreads();  // and every wave's reads are done: the caller may use LDS
}

// Workgroup b of a grid of at least `tiles` -> its tile, or -1: consecutive workgroups
// go round the 8 XCDs, each XCD takes a run of consecutive tiles
__device__ __forceinline__ int mx_xcd_tile(int b, int tiles) {
  const int xcd = b & 7, per = tiles >> 3, rem = tiles & 7;
  const int i = b >> 3;
  if (i >= per + (xcd < rem ? 1 : 0)) return -1;
  return xcd * per + min(xcd, rem) + i;
}
// How `count` rows fall into tiles of kBM: the last one takes the rest, and up to kOver
// rows more than kBM rather than leaving them a tile of their own.
template <int kBM, int kOver>
__host__ __device__ inline int mx_row_tiles(int count) {
  const int full = count / kBM, rest = count - full * kBM;
  return full + (rest > (full ? kOver : 0) ? 1 : 0);
}
// tile t of tiles_n x tiles_m, in groups of 8 token tiles (kept in one L2)
__device__ __forceinline__ void mx_tile_at(int t, int tiles_n, int tiles_m, int& tn, int& tm) {
  const int group = t / (8 * tiles_n);
  const int m0 = group * 8, gm = min(8, tiles_m - m0);
  const int in = t - group * 8 * tiles_n;
  tm = m0 + in % gm;
  tn = in / gm;
}

// Outputs through LDS, so that they leave as whole lines, 16 bytes a lane: kCols values of
// type T a token (fp32, 7414 x 2049 x 941 with its quantisation 29 us, straight from the
// registers 33). Each wave takes its token tiles in turn through its own kMxStage bytes (rows padded by 16 bytes); put(t, o)
// writes the lane's values of token tile t at its token's place o; row_of(i) gives where the
// outputs of the wave's token i start, or NULL.
template <typename T, int kCols>
constexpr int kMxStage = 32 * (kCols * sizeof(T) + 16);

template <typename T, int kT, int kCols, typename Put, typename Row>
__device__ __forceinline__ void mx_store(uint8_t* lds, Put put, Row row_of, int n_left) {
  typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
  constexpr int kPer = 16 / sizeof(T);  // values a lane
  constexpr int kPitch = kCols * sizeof(T) + 16, kLanes = kCols / kPer, kRows = 64 / kLanes;
  static_assert(kLanes <= 64 && kRows <= 32, "whole rows a wave");
  const int lane = threadIdx.x & 63;
  uint8_t* o = lds + (threadIdx.x >> 6) * kMxStage<T, kCols>;
  const int c16 = lane % kLanes, left = n_left - kPer * c16;
  const auto in_order = [] {  // a wave's LDS accesses stay in order, in the code as well
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    put(t, o + (lane & 31) * kPitch);
    in_order();
    u32x4_t v[32 / kRows];
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i)
      v[i] = *reinterpret_cast<const u32x4_t*>(o + (i * kRows + lane / kLanes) * kPitch + 16 * c16);
    in_order();
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      T* to = row_of(t * 32 + i * kRows + lane / kLanes);
      if (!to) continue;
      to += kPer * c16;
      if (left >= kPer) {
        *reinterpret_cast<u32x4_any_t*>(to) = v[i];
      } else {
#pragma unroll
        for (int c = 0; c < kPer - 1; ++c) {
          if (c >= left) continue;
          if constexpr (sizeof(T) == 2)
            to[c] = static_cast<T>(v[i][c >> 1] >> (16 * (c & 1)));
          else
            to[c] = __uint_as_float(v[i][c]);
        }
      }
    }
  }
}

// a tile's outputs: this wave's weight rows in order
template <typename T, int kT, typename Row>
__device__ __forceinline__ void mx_store_tile(uint8_t* lds, const f32x16_t (&acc)[kQ][kT], Row row_of,
                                              int n_left) {
  const int hi = (threadIdx.x & 63) >> 5;
  mx_store<T, kT, 32 * kQ>(
      lds,
      [&](int t, uint8_t* o) {
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x16_t& d = acc[q][t];
            uint8_t* to = o + (q * 32 + j * 8 + 4 * hi) * sizeof(T);
            if constexpr (sizeof(T) == 2)
              *reinterpret_cast<u32x2_t*>(to) =
                  u32x2_t{mx_bf16x2(d[4 * j], d[4 * j + 1]), mx_bf16x2(d[4 * j + 2], d[4 * j + 3])};
            else
              *reinterpret_cast<f32x4_t*>(to) = f32x4_t{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]};
          }
      },
      row_of, n_left);
}

}  // namespace moeblk
