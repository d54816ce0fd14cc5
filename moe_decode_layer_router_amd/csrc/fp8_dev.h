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
constexpr int kCpolNt = 2;  // cache-policy operand of the buffer intrinsics: non-temporal

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
// Fast: one e4m3 MFMA, at twice the bf16 rate. Of every 8 products with adjacent K it
// keeps multiples of 2^(E - 13), E the largest sum of two operands' exponent fields
// among the 8 (measured: beside 448 x 448, with E = 16, a product of 8 is kept and one
// of 4 lost; a subnormal has the field of 2^-6); the 16 sums of 8 are then added to
// about 24 bits. A group loses less than 7 x 2^(E - 13): of normal values at most
// 2^-10 of the sum of magnitudes, however much of that cancels (1.6 million random
// blocks: of normally distributed values at most 2.6e-5 of it, of values over 16 binades
// 2.8e-4). In the 2-norm a block of normally distributed values comes out 1.5e-5 off, with
// the 16x16x32 and 32x32x64 e4m3 MFMAs alike.
//
// Every memory-bound kernel takes the exact form. The fast one is for products of many
// rows with bf16 outputs, where the matrix rate counts (fp8.hip, exact_sums); the sum
// over blocks is fp32 in both forms.
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
// amax's exponent less 8, plus one where its mantissa is above 1.75.
__device__ __forceinline__ float fp8_block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int f = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // e + 127
  f = f < 1 ? 1 : f;
  return __uint_as_float((u >> 23) >= 255u ? 0x7fc00000u : static_cast<uint32_t>(f) << 23);
}

// four outputs of a row at element `at`, `left` of them inside the row; kFp32: fp32
// outputs are possible. Stores of four take any alignment (rows of any length).
template <bool kFp32>
__device__ __forceinline__ void store4(void* out, size_t at, int left, f32x4_t v, bool bf16) {
  typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));
  typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
  if (left <= 0) return;
  if (!kFp32 || bf16) {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    const u32x2_t p = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    if (left >= 4) {
      *reinterpret_cast<u32x2_any_t*>(o) = p;
    } else {
      o[0] = static_cast<uint16_t>(p[0]);
      if (left > 1) o[1] = static_cast<uint16_t>(p[0] >> 16);
      if (left > 2) o[2] = static_cast<uint16_t>(p[1]);
    }
  } else {
    float* o = static_cast<float*>(out) + at;
    if (left >= 4) {
      *reinterpret_cast<f32x4_any_t*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) o[i] = v[i];
    }
  }
}

// ---------------------------------------------------------------- K parts
//
// A product with too few tiles to fill the CUs is split over K: `parts`
// workgroups a tile, each leaving its fp32 sums in memory; the last of a tile to
// finish adds them in part order (deterministic) and writes the output. Sums are
// stored through to memory (a device-scope release would write back the
// whole L2), counted once every thread's stores are done, and loaded through.
struct SplitK {
  int parts;
  int32_t* counters;  // one a tile, zero between calls
  f32x4_t* sums;      // [tile][part][kN][threads]
};

constexpr int kSplitTiles = 256;                        // most tiles that are split
constexpr size_t kSplitCounterBytes = 256 * kSplitTiles;  // 256 bytes apart: a line each

__device__ __forceinline__ void store16_through(f32x4_t* p, f32x4_t v) {
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  typedef uint64_t u64x2_t __attribute__((ext_vector_type(2)));
  const u64x2_t u = __builtin_bit_cast(u64x2_t, v);
  __hip_atomic_store(q, u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(q + 1, u[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4_t load16_through(f32x4_t* p) {
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  typedef uint64_t u64x2_t __attribute__((ext_vector_type(2)));
  const u64x2_t u = {__hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                     __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
  return __builtin_bit_cast(f32x4_t, u);
}

// v: this thread's kN sums of part p of tile `tile` (threads with `on`). True in
// the workgroup that holds the tile's totals afterwards. Every thread of the
// workgroup calls it; `last` is a word of LDS that nothing else uses by then.
template <int kN>
__device__ __forceinline__ bool join_parts(const SplitK& k, int tile, int p, bool on,
                                           f32x4_t (&v)[kN], int* last) {
  if (k.parts == 1) return true;
  f32x4_t* t = k.sums + static_cast<size_t>(tile) * k.parts * kN * blockDim.x + threadIdx.x;
  if (on) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      store16_through(t + (static_cast<size_t>(p) * kN + i) * blockDim.x, v[i]);
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) {
    int32_t* c = k.counters + tile * 64;
    *last = __hip_atomic_fetch_add(c, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == k.parts - 1;
    if (*last) __hip_atomic_store(c, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!*last) return false;
  if (on) {
    constexpr int kBatch = kN >= 16 ? 1 : 16 / kN > 8 ? 8 : 16 / kN;  // parts loaded together
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = f32x4_t{0, 0, 0, 0};
    for (int q = 0; q < k.parts; q += kBatch) {
      f32x4_t u[kBatch][kN];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int i = 0; i < kN; ++i)
          u[j][i] = load16_through(t + (static_cast<size_t>(min(q + j, k.parts - 1)) * kN + i) *
                                           blockDim.x);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (q + j < k.parts) v[i] += u[j][i];
    }
  }
  return true;
}

// blocks [kb0, kb1) of part p
__device__ __forceinline__ void part_range(int Kb, int parts, int p, int& kb0, int& kb1) {
  kb0 = static_cast<int>(static_cast<int64_t>(Kb) * p / parts);
  kb1 = static_cast<int>(static_cast<int64_t>(Kb) * (p + 1) / parts);
}

}  // namespace moeblk
