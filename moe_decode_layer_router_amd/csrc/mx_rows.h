// mx_rows.h -- the MXFP4 product of few rows: weights straight into registers
// (device code).
//
// A workgroup takes a block of 64 weight rows x 16 kTT rows (tokens); its kNW waves take
// every kNW-th 128-K chunk of the workgroup's part, kRing chunks' loads in flight each. The
// waves' sums are added through LDS in wave order. The weights are read once per group of
// tokens, and their bytes bound the call.
//
// kSrc: quantised rows, or the rows themselves: a lane holds one MX block of its token, 32
// adjacent columns, so it quantises them by itself, without a launch in front and with the
// values moe_mx_quant gives.
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
  constexpr bool kF32 = kSrc == kMxRowsFp32;
  constexpr int kPer = kF32 ? 4 : 8;  // columns 16 bytes hold
  const uint8_t* p = static_cast<const uint8_t*>(row) + static_cast<size_t>(c0) * (kF32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < MxRaw<kSrc>::kWords / 4; ++i) {
    u32x4_t q = {0, 0, 0, 0};
    if (kPer * (i + 1) <= left) q = *reinterpret_cast<const mx_u32x4_any_t*>(p + 16 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v.w[4 * i + j] = q[j];
  }
  if (left <= 0 || left >= 32 || left % kPer == 0) return;
  // the row ends inside 16 bytes: their columns one by one, the last one in the place of
  // those behind it (all loads at once, none outside the row), which are then cleared
  const int first = left / kPer * kPer;
  uint32_t t[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = min(first + j, left - 1);
    t[j] = kF32 ? reinterpret_cast<const uint32_t*>(p)[c] : reinterpret_cast<const uint16_t*>(p)[c];
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) t[j] = first + j < left ? t[j] : 0u;
#pragma unroll
  for (int i = 0; i < MxRaw<kSrc>::kWords / 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = kF32 ? t[j] : t[2 * j % kPer] | (t[(2 * j + 1) % kPer] << 16);
      v.w[4 * i + j] = first == kPer * i ? w : v.w[4 * i + j];
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

// What a workgroup multiplies: chunks [c0, c1) of the row block whose first tile is at w, and
// of tokens t0 .. t0 + 16 kTT - 1 of M.
struct MxRowsTile {
  const uint8_t* w;
  int Kc, c0, c1;
  int t0, M;
};

template <int kTT, int kNW>
constexpr int mx_rows_red() {
  return kNW * (4 * kTT < kNW ? 4 * kTT : kNW) * 64;
}

// sum[e]: of tile i = kNW e + wave, i < 4 kTT: row tile i / kTT, token tile i % kTT. red:
// mx_rows_red elements. row_of(token) gives a token's row of x.
template <int kTT, int kNW, int kRing, int kSrc, typename F>
__device__ __forceinline__ void mx_rows_body(const MxRowsTile& p, const void* x, int K,
                                             const uint8_t* xq, const uint8_t* xs, F row_of,
                                             f32x4_t* red, f32x4_t (&sum)[(4 * kTT + kNW - 1) / kNW]) {
  constexpr int kRT = 4;
  constexpr bool kRaw = kSrc != kMxRowsQ;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int Kc = p.Kc;
  const uint8_t *xp[kTT], *sp[kTT];
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    const size_t row = row_of(min(p.t0 + 16 * t + m16, p.M - 1));
    if constexpr (kRaw) {
      xp[t] = static_cast<const uint8_t*>(x) + row * K * (kSrc == kMxRowsFp32 ? 4 : 2);
    } else {
      xp[t] = xq + row * (static_cast<size_t>(Kc) * 64) + 16 * g;
      sp[t] = xs + row * (static_cast<size_t>(Kc) * 4) + g;
    }
  }
  u32x4_t w[kRing][kRT], b[kRaw ? 1 : kRing][kTT];
  uint32_t sw[kRing], sb[kRaw ? 1 : kRing][kTT];
  MxRaw<kSrc> v[kRaw ? kRing : 1][kRaw ? kTT : 1];
  const auto load = [&](int i, int c) {
    const uint8_t* t = p.w + static_cast<size_t>(c) * kMxTileBytes;
#pragma unroll
    for (int r = 0; r < kRT; ++r) w[i][r] = ld_nt<u32x4_t>(t + r * 1024 + lane * 16);
    sw[i] = *reinterpret_cast<const uint32_t*>(t + 4096 + lane * 4);
#pragma unroll
    for (int q = 0; q < kTT; ++q) {
      if constexpr (kRaw) {
        const int col = kChunkK * c + kMxBlock * g;
        mx_load_raw<kSrc>(xp[q], col, K - col, v[i][q]);
      } else {
        b[i][q] = *reinterpret_cast<const u32x4_t*>(xp[q] + c * 64);
        sb[i][q] = sp[q][c * 4];
      }
    }
  };
  f32x4_t acc[kRT][kTT];
#pragma unroll
  for (int r = 0; r < kRT; ++r)
#pragma unroll
    for (int t = 0; t < kTT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
  const auto multiply = [&](int i) {
    const int j = kRaw ? 0 : i;
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      if constexpr (kRaw) b[0][t] = mx_quant32<kSrc>(v[i][t], sb[0][t]);
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
