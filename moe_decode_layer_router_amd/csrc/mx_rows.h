// mx_rows.h -- the MXFP4 product of few rows: weights straight into registers
// (device code).
//
// A workgroup takes a block of 64 weight rows x 16 kTT rows (tokens); its kNW waves take
// every kNW-th 128-K chunk of the workgroup's part, kRing chunks' loads in flight each. The
// waves' sums are added through LDS in wave order. The weights are read once per group of
// tokens, and their bytes bound the call.
//
// kSrc: quantised rows, or the rows themselves, quantised here without a launch in front and
// to the values moe_mx_quant gives: 16 lanes read a row's chunk (whole lines; a block a lane,
// 64 bytes apart, touches each line four times: 99 x 286 x 1899 14.1 us, so 10.4), four of
// them share a block, and the codes pass through the wave's own LDS into operand order.
#pragma once

#include "fp8_quant.h"
#include "mx_dev.h"

namespace moeblk {

enum MxSource { kMxRowsBf16, kMxRowsFp32, kMxRowsQ };

typedef u32x4_t mx_u32x4_any_t __attribute__((aligned(2)));

// 8 columns of a row, as 8 fp32 words or 4 pairs of bf16
template <int kSrc>
struct MxRaw {
  uint32_t w[kSrc == kMxRowsFp32 ? 8 : 4];
};

// Columns c .. c + 7 of a row of K; where the row ends before that, its last 8 columns, for
// mx_shift_raw to put in place. Rows of fewer than 8 columns come with their zeros.
template <int kSrc>
__device__ __forceinline__ void mx_load_raw(const void* row, int c, int K, MxRaw<kSrc>& v) {
  constexpr bool kF32 = kSrc == kMxRowsFp32;
  const uint8_t* p = static_cast<const uint8_t*>(row);
  if (K >= 8) {
    p += static_cast<size_t>(min(c, K - 8)) * (kF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (kF32 ? 2 : 1); ++i) {
      const u32x4_t q = *reinterpret_cast<const mx_u32x4_any_t*>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.w[4 * i + j] = q[j];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < (kF32 ? 8 : 4); ++j) v.w[j] = 0;
#pragma unroll
  for (int j = 0; j < 7; ++j) {
    if (c + j >= K) continue;
    if constexpr (kF32)
      v.w[j] = reinterpret_cast<const uint32_t*>(p)[c + j];
    else
      v.w[j >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[c + j]) << (16 * (j & 1));
  }
}

// the columns `by` places further on in front, zeros behind them
template <int kSrc>
__device__ __forceinline__ void mx_shift_raw(MxRaw<kSrc>& v, int by) {
  by = min(by, 8);
  if constexpr (kSrc == kMxRowsFp32) {
#pragma unroll
    for (int s = 4; s >= 1; s >>= 1) {
      const bool on = (by & s) != 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) v.w[i] = on ? (i + s < 8 ? v.w[i + s] : 0u) : v.w[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i] = by == 8 ? 0u : v.w[i];
  } else {
    uint64_t lo = v.w[0] | static_cast<uint64_t>(v.w[1]) << 32, hi = v.w[2] | static_cast<uint64_t>(v.w[3]) << 32;
    if (by & 4) lo = hi, hi = 0;
    const int s = 16 * (by & 3);
    lo = s ? (lo >> s) | (hi << (64 - s)) : lo;
    hi >>= s;
    if (by == 8) lo = hi = 0;
    v.w[0] = static_cast<uint32_t>(lo);
    v.w[1] = static_cast<uint32_t>(lo >> 32);
    v.w[2] = static_cast<uint32_t>(hi);
    v.w[3] = static_cast<uint32_t>(hi >> 32);
  }
}

// The codes of 8 columns by one of four adjacent lanes that share a block (all of which
// take part), and the block's scale byte.
template <int kSrc>
__device__ __forceinline__ uint32_t mx_quant8(const MxRaw<kSrc>& v, uint32_t& byte) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  uint32_t m = 0;
  if constexpr (kSrc == kMxRowsFp32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v.w[i] & 0x7fffffffu);
  } else {
    u16x2_t p = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, v.w[i] & 0x7fff7fffu));
    m = static_cast<uint32_t>(p[0] > p[1] ? p[0] : p[1]) << 16;
  }
  m = max_dpp<0xb1>(m);  // lane ^ 1
  m = max_dpp<0x4e>(m);  // lane ^ 2
  byte = mx_scale_byte(m);
  const float s = e8m0_scale(byte);
  uint32_t q;
  if constexpr (kSrc == kMxRowsFp32) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v.w[i]);
    q = mx_codes(f, s);
  } else {
    q = mx_codes_bf16(v.w, s);
  }
  return mx_codes_or_zero(q, byte);
}

constexpr int kMxPass = 1024 + 64;  // LDS bytes of a wave's token tile: codes, scale bytes

// What a workgroup multiplies: chunks [c0, c1) of the row block whose first tile is at w, and
// of tokens t0 .. t0 + 16 kTT - 1 of M.
struct MxRowsTile {
  const uint8_t* w;
  int Kc, c0, c1;
  int t0, M;
};

template <int kTT, int kNW>
constexpr int mx_rows_red = kNW * 4 * kTT * 64;

// sum: of tile i = wave < 4 kTT: row tile i / kTT, token tile i % kTT. red:
// mx_rows_red elements; pass: kNW kTT kMxPass bytes (rows as they are only). row_of(token)
// gives a token's row of x.
template <int kTT, int kNW, int kRing, int kSrc, typename F>
__device__ __forceinline__ void mx_rows_body(const MxRowsTile& p, const void* x, int K,
                                             const uint8_t* xq, const uint8_t* xs, F row_of,
                                             uint8_t* pass, f32x4_t* red, f32x4_t& sum) {
  constexpr int kRT = 4, kTiles = kRT * kTT;
  static_assert(kTiles <= kNW, "a tile a wave");
  constexpr bool kRaw = kSrc != kMxRowsQ;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int Kc = p.Kc;
  constexpr int kRows = kRaw ? 4 : 1;  // rows a lane reads of a token tile
  const int tokens = p.M - p.t0;
  const uint8_t *xp[kTT][kRows], *sp[kTT];
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const size_t row = row_of(min(p.t0 + 16 * t + (kRaw ? 4 * i + g : m16), p.M - 1));
      if constexpr (kRaw) {
        xp[t][i] = static_cast<const uint8_t*>(x) + row * K * (kSrc == kMxRowsFp32 ? 4 : 2);
      } else {
        xp[t][i] = xq + row * (static_cast<size_t>(Kc) * 64) + 16 * g;
        sp[t] = xs + row * (static_cast<size_t>(Kc) * 4) + g;
      }
    }
  }
  u32x4_t w[kRing][kRT], b[kRaw ? 1 : kRing][kTT];
  uint32_t sw[kRing], sb[kRaw ? 1 : kRing][kTT];
  MxRaw<kSrc> v[kRaw ? kRing : 1][kTT][kRows];
  const auto load = [&](int i, int c) {
    const uint8_t* t = p.w + static_cast<size_t>(c) * kMxTileBytes;
#pragma unroll
    for (int r = 0; r < kRT; ++r) w[i][r] = ld_nt<u32x4_t>(t + r * 1024 + lane * 16);
    sw[i] = *reinterpret_cast<const uint32_t*>(t + 4096 + lane * 4);
#pragma unroll
    for (int q = 0; q < kTT; ++q) {
      if constexpr (kRaw) {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (16 * q + 4 * j < tokens) mx_load_raw<kSrc>(xp[q][j], kChunkK * c + 8 * m16, K, v[i][q][j]);
      } else {
        b[i][q] = *reinterpret_cast<const u32x4_t*>(xp[q][0] + c * 64);
        sb[i][q] = sp[q][c * 4];
      }
    }
  };
  f32x4_t acc[kRT][kTT];
#pragma unroll
  for (int r = 0; r < kRT; ++r)
#pragma unroll
    for (int t = 0; t < kTT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
  const auto multiply = [&](int i, int c) {
    const int j = kRaw ? 0 : i;
    const bool tail = kRaw && K >= 8 && kChunkK * (c + 1) > K;
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      if constexpr (kRaw) {
        // row 4 j + g, columns 8 m16 .. + 7 -> token m16, block g; a wave's LDS accesses stay
        // in order, in the code as well
        uint8_t* o = pass + (wave * kTT + t) * kMxPass;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (16 * t + 4 * j >= tokens) break;  // nothing there; those tokens' sums are not looked at
          if (tail) mx_shift_raw<kSrc>(v[i][t][j], kChunkK * c + 8 * m16 - min(kChunkK * c + 8 * m16, K - 8));
          uint32_t byte;
          const uint32_t q = mx_quant8<kSrc>(v[i][t][j], byte);
          *reinterpret_cast<uint32_t*>(o + (4 * j + g) * 64 + 4 * m16) = q;
          if ((m16 & 3) == 0) o[1024 + (4 * j + g) * 4 + (m16 >> 2)] = static_cast<uint8_t>(byte);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        b[0][t] = *reinterpret_cast<const u32x4_t*>(o + m16 * 64 + g * 16);
        sb[0][t] = o[1024 + m16 * 4 + g];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int r = 0; r < kRT; ++r)
        acc[r][t] = mfma_mx_row(r, w[i][r], b[j][t], acc[r][t], sw[i], sb[j][t]);
    }
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i)
    if (p.c0 + wave + kNW * i < p.c1) load(i, p.c0 + wave + kNW * i);
  for (int base = p.c0 + wave; base < p.c1; base += kNW * kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      const int c = base + kNW * i;
      if (c < p.c1) {
        multiply(i, c);
        if (c + kNW * kRing < p.c1) load(i, c + kNW * kRing);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) red[(wave * kTiles + i) * 64 + lane] = acc[i / kTT][i % kTT];
  __syncthreads();
  sum = f32x4_t{0, 0, 0, 0};
  if (wave < kTiles) {
    sum = red[wave * 64 + lane];
#pragma unroll
    for (int q = 1; q < kNW; ++q) sum += red[(q * kTiles + wave) * 64 + lane];
  }
}

}  // namespace moeblk
