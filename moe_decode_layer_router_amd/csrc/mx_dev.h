// mx_dev.h -- device code shared by the MXFP4 (e2m1 values, an e8m0 scale per 32)
// kernels for many rows.
//
// Rows are held canonically: codes [M][Kc * 64] (two a byte, the even column in the
// low nibble), scale bytes [M][Kc * 4], Kc = ceil(K / 128) chunks. Weights are the
// tiles of common.h (64 rows x 128 K, 4352 bytes), so the experts' weights of the
// decode path serve here as they are. A lane's 16 bytes of either operand are one MX
// block, which is what the 16x16x128 scaled MFMA takes: lane (row or token l % 16,
// block l / 16), one scale byte a lane.
//
// That MFMA's sums are fp32 sums: measured over random codes and scales of 2^-27 ..
// 2^27 against fp64, at most 2^-22.5 of the sum of magnitudes off, and exact where all
// products fit 24 bits (two cancelling products of 36 x 2^14 beside ordinary ones
// included); products of e2m1 values are multiples of 1/4 up to 36.
#pragma once

#include "common.h"
#include "fp8_dev.h"

namespace moeblk {

constexpr int kMxBlock = 32;  // values a scale covers
constexpr int kMxNan = 255;   // scale byte of a block that is not finite

__host__ __device__ inline int mx_chunks(int K) { return (K + kChunkK - 1) / kChunkK; }
__host__ __device__ inline int mx_row_blocks(int N) {
  return (N + kRowsPerBlock - 1) / kRowsPerBlock;
}
__host__ __device__ inline size_t mx_packed_bytes(int N, int K) {
  return static_cast<size_t>(mx_row_blocks(N)) * mx_chunks(K) * kMxTileBytes;
}

// D[16x16] += A[16x128] B[128x16], e2m1 in, scales from byte kA / kB of sa / sb
template <int kA, int kB>
__device__ __forceinline__ f32x4_t mfma_mx(u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa,
                                           uint32_t sb) {
  const i32x8_t a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, kA, (int)sa, kB,
                                                          (int)sb);
}
// row tile r's scale byte chosen at compile time after unrolling
__device__ __forceinline__ f32x4_t mfma_mx_row(int r, u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa,
                                               uint32_t sb) {
  switch (r & 3) {
    case 0: return mfma_mx<0, 0>(a, b, c, sa, sb);
    case 1: return mfma_mx<1, 0>(a, b, c, sa, sb);
    case 2: return mfma_mx<2, 0>(a, b, c, sa, sb);
    default: return mfma_mx<3, 0>(a, b, c, sa, sb);
  }
}

// The scale byte of a block whose largest magnitude has these fp32 bits: e + 127 with
// the smallest e >= -127 such that amax < 7 2^e, so that every value rounds to at
// most 6 2^e (7 lies halfway between 6 and 8) and none saturates. 7 = 1.75 2^2: the
// exponent field less 2, plus one where the mantissa is 1.75 or more.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kMxNan;
  const int e = static_cast<int>((amax + 0x200000u) >> 23) - 2;
  return static_cast<uint32_t>(e < 0 ? 0 : e);
}
// a block that is not finite gets zero codes beside its NaN scale
__device__ __forceinline__ uint32_t mx_codes_or_zero(uint32_t codes, uint32_t byte) {
  return byte == kMxNan ? 0u : codes;
}

// 8 values -> 8 codes, the first in the low nibble; division by the scale is part of
// the converts and exact, they round to nearest even
__device__ __forceinline__ uint32_t mx_codes(const float (&v)[8], float scale) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
  return q;
}
// 8 bf16 values in 4 words
__device__ __forceinline__ uint32_t mx_codes_bf16(const uint32_t* w, float scale) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, w[0]), scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, w[1]), scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, w[2]), scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, w[3]), scale, 3);
  return q;
}

// two fp32 -> bf16 in a word, to nearest even (one instruction)
__device__ __forceinline__ uint32_t mx_bf16x2(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

// silu(g) u in fp32; exp(-|g|) never overflows. The exponential is the hardware's of a rounded
// product: for g < 0 it is off by |g| 2^-24 of the result, 2^-17 at g = -100, where half a step of
// bf16 is 2^-9 and of e2m1 2^-3 (the decode path, bound by its weights, evaluates it in fp64).
__device__ __forceinline__ float mx_swiglu(float g, float u) {
  const float e = __expf(-fabsf(g));
  return (g >= 0.0f ? g : g * e) / (1.0f + e) * u;
}

}  // namespace moeblk
