// mx_rows.h -- the MXFP4 product of few rows: weights straight into registers
// (device code).
//
// A workgroup takes 16 kRT weight rows x 16 kTT rows (tokens); its kNW waves take
// every kNW-th 128-K chunk of the workgroup's part, kRing chunks' loads in flight
// each. The waves' sums are added through LDS in wave order. The weights are read once
// per group of tokens, and their bytes bound the call.
//
// kSrc: quantised rows, or (up to 16 rows) the rows themselves: a lane holds one
// MX block of its token, 32 adjacent columns, so it quantises them by itself, without
// a launch in front and with the values moe_mx_quant gives.
#pragma once

#include "mx_dev.h"

namespace moeblk {

enum MxSource { kMxRowsBf16, kMxRowsFp32, kMxRowsQ };

typedef u32x4_t mx_u32x4_any_t __attribute__((aligned(2)));

// 32 columns of a row from column c0 on (`left` of them inside the row), as fp32 words
// or pairs of bf16
template <int kSrc>
struct MxRaw {
  static constexpr int kWords = kSrc == kMxRowsFp32 ? 32 : 16;
  uint32_t w[kWords];
};

template <int kSrc>
__device__ __forceinline__ void mx_load_raw(const void* row, int c0, int left, MxRaw<kSrc>& v) {
  constexpr int kPer = kSrc == kMxRowsFp32 ? 4 : 8;  // columns 16 bytes hold
#pragma unroll
  for (int i = 0; i < MxRaw<kSrc>::kWords / 4; ++i) {
    u32x4_t q = {0, 0, 0, 0};
    const int c = kPer * i;
    if constexpr (kSrc == kMxRowsFp32) {
      const float* p = static_cast<const float*>(row) + c0 + c;
      if (c + kPer <= left) {
        q = *reinterpret_cast<const mx_u32x4_any_t*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (c + j < left) q[j] = __float_as_uint(p[j]);
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(row) + c0 + c;
      if (c + kPer <= left) {
        q = *reinterpret_cast<const mx_u32x4_any_t*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (c + j < left) q[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v.w[4 * i + j] = q[j];
  }
}

// a block's 32 codes, and its scale byte
template <int kSrc>
__device__ __forceinline__ u32x4_t mx_quant32(const MxRaw<kSrc>& v, uint32_t& byte) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  uint32_t m = 0;
  if constexpr (kSrc == kMxRowsFp32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t a = v.w[i] & 0x7fffffffu;
      m = m > a ? m : a;
    }
  } else {
    u16x2_t p = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, v.w[i] & 0x7fff7fffu));
    m = static_cast<uint32_t>(p[0] > p[1] ? p[0] : p[1]) << 16;
  }
  byte = mx_scale_byte(m);
  const float s = e8m0_scale(byte);
  u32x4_t q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kSrc == kMxRowsFp32) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v.w[8 * i + j]);
      q[i] = mx_codes(f, s);
    } else {
      q[i] = mx_codes_bf16(&v.w[4 * i], s);
    }
    q[i] = mx_codes_or_zero(q[i], byte);
  }
  return q;
}

// What a workgroup multiplies: chunks [c0, c1) of 16 kRT weight rows (from row tile
// rt0 of the matrix at w on) and of tokens t0 .. t0 + 16 kTT - 1 of M.
struct MxRowsTile {
  const uint8_t* w;
  int rt0, Kc, c0, c1;
  int t0, M;
};

template <int kRT, int kTT, int kNW>
constexpr int mx_rows_red() {
  return kNW * (kRT * kTT < kNW ? kRT * kTT : kNW) * 64;
}

// sum[e]: of tile i = kNW e + wave, i < kRT kTT: row tile i / kTT, token tile i % kTT.
// red: mx_rows_red elements. row_of(token) gives a token's row of x.
template <int kRT, int kTT, int kNW, int kRing, int kSrc, typename F>
__device__ __forceinline__ void mx_rows_body(const MxRowsTile& p, const void* x, int K,
                                             const uint8_t* xq, const uint8_t* xs, F row_of,
                                             f32x4_t* red, f32x4_t (&sum)[(kRT * kTT + kNW - 1) / kNW]) {
  static_assert(kRT == 1 || kRT == 2 || kRT == 4, "row tiles of one row block");
  static_assert(kSrc == kMxRowsQ || kTT == 1, "at most 16 rows are quantised here");
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int Kc = p.Kc, r0 = p.rt0 & 3;
  const uint8_t* wt = p.w + static_cast<size_t>(p.rt0 >> 2) * Kc * kMxTileBytes;
  const uint8_t *xp[kTT], *sp[kTT];
  const void* raw = nullptr;
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    const size_t row = row_of(min(p.t0 + 16 * t + m16, p.M - 1));
    if constexpr (kSrc == kMxRowsQ) {
      xp[t] = xq + row * (static_cast<size_t>(Kc) * 64) + 16 * g;
      sp[t] = xs + row * (static_cast<size_t>(Kc) * 4) + g;
    } else {
      raw = static_cast<const uint8_t*>(x) + row * K * (kSrc == kMxRowsFp32 ? 4 : 2);
    }
  }
  u32x4_t w[kRing][kRT], b[kRing][kTT];
  uint32_t sw[kRing], sb[kRing][kTT];
  MxRaw<kSrc> v[kSrc == kMxRowsQ ? 1 : kRing];
  const auto load = [&](int i, int c) {
    const uint8_t* t = wt + static_cast<size_t>(c) * kMxTileBytes;
#pragma unroll
    for (int r = 0; r < kRT; ++r) w[i][r] = ld_nt<u32x4_t>(t + (r0 + r) * 1024 + lane * 16);
    sw[i] = *reinterpret_cast<const uint32_t*>(t + 4096 + lane * 4);
    if constexpr (kSrc == kMxRowsQ) {
#pragma unroll
      for (int t = 0; t < kTT; ++t) {
        b[i][t] = *reinterpret_cast<const u32x4_t*>(xp[t] + c * 64);
        sb[i][t] = sp[t][c * 4];
      }
    } else {
      const int col = kChunkK * c + kMxBlock * g;
      mx_load_raw<kSrc>(raw, col, K - col, v[i]);
    }
  };
  f32x4_t acc[kRT][kTT];
#pragma unroll
  for (int r = 0; r < kRT; ++r)
#pragma unroll
    for (int t = 0; t < kTT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
  const auto multiply = [&](int i) {
    if constexpr (kSrc != kMxRowsQ) b[i][0] = mx_quant32<kSrc>(v[i], sb[i][0]);
    const uint32_t s = kRT == 4 ? sw[i] : sw[i] >> (8 * r0);
#pragma unroll
    for (int r = 0; r < kRT; ++r)
#pragma unroll
      for (int t = 0; t < kTT; ++t) acc[r][t] = mfma_mx_row(r, w[i][r], b[i][t], acc[r][t], s, sb[i][t]);
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i)
    if (p.c0 + wave + kNW * i < p.c1) load(i, p.c0 + wave + kNW * i);
  for (int base = p.c0 + wave; base < p.c1; base += kNW * kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      const int c = base + kNW * i;
      if (c < p.c1) {
        multiply(i);
        if (c + kNW * kRing < p.c1) load(i, c + kNW * kRing);
      }
    }
  }
  constexpr int kEach = (kRT * kTT + kNW - 1) / kNW;
  constexpr int kRound = kRT * kTT < kNW ? kRT * kTT : kNW;  // tiles a round
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (e) __syncthreads();
#pragma unroll
    for (int i = 0; i < kNW && e * kNW + i < kRT * kTT; ++i)
      red[(wave * kRound + i) * 64 + lane] = acc[(e * kNW + i) / kTT][(e * kNW + i) % kTT];
    __syncthreads();
    sum[e] = f32x4_t{0, 0, 0, 0};
    if (e * kNW + wave < kRT * kTT) {
      sum[e] = red[wave * 64 + lane];
#pragma unroll
      for (int q = 1; q < kNW; ++q) sum[e] += red[(q * kRound + wave) * 64 + lane];
    }
  }
}

}  // namespace moeblk
