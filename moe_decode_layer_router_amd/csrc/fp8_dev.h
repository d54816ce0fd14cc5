// fp8_dev.h -- device code shared by the FP8 (e4m3, block-128 scales) kernels.
//
// Packed FP8 weight, one N x K matrix (Kb = ceil(K / 128) K blocks, rows and
// columns padded with zeros): row tiles of 16 rows x K blocks of 128, one tile
// (rt, kb) 2048 contiguous bytes at (rt * Kb + kb) * 2048:
//   [h * 1024 + lane * 16, +16)  row m = lane % 16 of the tile at
//                                K = 128 kb + 32 (lane / 16) + 16 h .. + 16,
// so that a wave reads a 16 x 128 operand of the 16x16x128 MFMA as two
// contiguous 1 KiB loads. The row tiles are padded to a multiple of 4, then the
// fp32 scales [Nb][Kb] follow (Nb = ceil(N / 128)). The tokens' operand takes
// the same K order: lane (token l % 16, group l / 16) holds the 32 bytes at
// K = 128 kb + 32 (l / 16) of its row. (The order of K inside a block does not
// matter as long as both operands share it.)
#pragma once

#include "common.h"

namespace moeblk {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kFp8Block = 128;     // K (and weight rows) a scale covers
constexpr int kFp8TileBytes = 2048;  // 16 rows x 128 K
constexpr float kE4m3Max = 448.0f;

__host__ __device__ inline int fp8_kb(int K) { return (K + kFp8Block - 1) / kFp8Block; }
// row tiles, padded to whole blocks of 64 rows
__host__ __device__ inline int fp8_row_tiles(int N) { return (N + 63) / 64 * 4; }
__host__ __device__ inline size_t fp8_tile_bytes(int N, int K) {
  return static_cast<size_t>(fp8_row_tiles(N)) * fp8_kb(K) * kFp8TileBytes;
}
// a matrix's scales, padded to 16 bytes
__host__ __device__ inline size_t fp8_scale_bytes(int N, int K) {
  return (static_cast<size_t>((N + 127) / 128) * fp8_kb(K) * 4 + 15) / 16 * 16;
}
__host__ __device__ inline size_t fp8_packed_bytes(int N, int K) {
  return fp8_tile_bytes(N, K) + fp8_scale_bytes(N, K);
}

// One 128-K block product D[16x16] = A[16x128] B[128x16] from a zero accumulator
// (layout of D as in mfma_bf16), in two forms.
//
// Exact: the e4m3 values are converted to bf16 (which holds them all) and go
// through four bf16 MFMAs. Measured against fp64 on normal values: 9e-9 relative
// over a block, i.e. an fp32 sum.
//
// Fast: one e4m3 MFMA, at twice the bf16 rate. Its adder aligns the products
// to fewer bits than fp32 has: 1.5e-5 relative over a block on the same values
// (the 16x16x32 e4m3 MFMA and the 32x32x64 one alike). It is used where the
// result is rounded to bf16 (half a step is 3.9e-3) and matrix throughput
// bounds the call; the sum over blocks is fp32 in both forms.
__device__ __forceinline__ f32x4_t mfma_fp8_block(i32x8_t a, i32x8_t b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0, 0, 0, 0}, 0, 0, 0, 0, 0,
                                                          0);
}

// a lane's 32 e4m3 values as four bf16 MFMA operands
struct Bf16Frag {
  bf16x8_t v[4];
};

__device__ __forceinline__ Bf16Frag e4m3_to_bf16(i32x8_t a) {
  Bf16Frag f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[2 * q], 1.0f, false);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[2 * q], 1.0f, true);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[2 * q + 1], 1.0f, false);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[2 * q + 1], 1.0f, true);
    f.v[q] = bf16x8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
  return f;
}

__device__ __forceinline__ f32x4_t mfma_exact_block(const Bf16Frag& a, const Bf16Frag& b) {
  f32x4_t d = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q) d = mfma_bf16(a.v[q], b.v[q], d);
  return d;
}

__device__ __forceinline__ i32x8_t join8(u32x4_t lo, u32x4_t hi) {
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The scale of a block of magnitude `amax`: 2^e with the smallest e >= -126
// and amax <= 448 * 2^e; NaN if amax is not finite. 448 = 1.75 * 2^8, so e is
// amax's exponent less 8, plus one where its mantissa is above 1.75. `inv` = 1 / scale
// (exact; e <= 120, so it is a normal number).
__device__ __forceinline__ float fp8_block_scale(float amax, float& inv) {
  const uint32_t u = __float_as_uint(amax);
  int f = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // e + 127
  f = f < 1 ? 1 : f;
  if ((u >> 23) >= 255u) {
    inv = __uint_as_float(0x7fc00000u);
    return inv;
  }
  inv = __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
  return __uint_as_float(static_cast<uint32_t>(f) << 23);
}

// max of magnitudes that keeps a NaN (fmaxf would drop it): non-negative
// floats order as their bit patterns, NaNs above infinity
__device__ __forceinline__ float max_mag(float a, float b) {
  const uint32_t ua = __float_as_uint(a) & 0x7fffffffu, ub = __float_as_uint(b) & 0x7fffffffu;
  return __uint_as_float(ua > ub ? ua : ub);
}

// four fp32, each |v| <= 448 (or NaN), to e4m3, round to nearest even
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

}  // namespace moeblk
