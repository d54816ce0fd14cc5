// fp8_quant.h -- rows to e4m3 with a scale per 128 columns (device code).
//
// A (row, 128-column block) is 8 lanes of 16 columns: its magnitude maximum is
// three DPP steps, each lane stores 16 bytes. Division by the scale is part of
// the converts and exact (a power of two), so the only rounding is e4m3's.
// Magnitudes are compared as integers (non-negative floats order as their bit
// patterns, infinity and NaN last), two bf16 at a time.
#pragma once

#include "fp8_dev.h"

namespace moeblk {

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef int16_t i16x2_t __attribute__((ext_vector_type(2)));

template <typename T>
struct Raw16 {  // 16 columns of a row as loaded
  uint32_t w[4 * sizeof(T)];
};

// 16 bytes at an element's alignment: rows of any length start anywhere, and global
// loads of any width take any alignment
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));

template <typename T>
__device__ __forceinline__ void load16(const T* row, int c0, int K, Raw16<T>& v) {
  if (c0 + 16 <= K) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
      const u32x4_t q = *reinterpret_cast<const u32x4_any_t*>(row + c0 + 16 / sizeof(T) * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.w[4 * i + j] = q[j];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < static_cast<int>(4 * sizeof(T)); ++i) v.w[i] = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (c0 + i < K) {
      if constexpr (sizeof(T) == 2)
        v.w[i >> 1] |= static_cast<uint32_t>(row[c0 + i]) << (16 * (i & 1));
      else
        v.w[i] = __float_as_uint(row[c0 + i]);
    }
  }
}

template <int kCtrl>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xf, 0xf, false));
  return v > o ? v : o;
}

// 16 columns of a block by one of 8 adjacent lanes: the e4m3 values, and the
// block's scale (the same in all 8 lanes, which must all take part)
template <typename T>
__device__ __forceinline__ u32x4_t quant16(const Raw16<T>& v, float& scale) {
  uint32_t m;
  if constexpr (sizeof(T) == 2) {
    u16x2_t p = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, v.w[i] & 0x7fff7fffu));
    m = static_cast<uint32_t>(p[0] > p[1] ? p[0] : p[1]) << 16;
  } else {
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = v.w[i] & 0x7fffffffu;
      m = m > a ? m : a;
    }
  }
  m = max_dpp<0xb1>(m);   // lane ^ 1
  m = max_dpp<0x4e>(m);   // lane ^ 2
  m = max_dpp<0x141>(m);  // the mirror within 8 lanes: the other four
  scale = fp8_block_scale(__uint_as_float(m));
  u32x4_t q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    i16x2_t r = {0, 0};
    if constexpr (sizeof(T) == 2) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, v.w[2 * i]),
                                                    scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, v.w[2 * i + 1]),
                                                    scale, true);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(v.w[4 * i]),
                                                   __uint_as_float(v.w[4 * i + 1]), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(v.w[4 * i + 2]),
                                                   __uint_as_float(v.w[4 * i + 3]), scale, true);
    }
    q[i] = __builtin_bit_cast(uint32_t, r);
  }
  return q;
}

}  // namespace moeblk
