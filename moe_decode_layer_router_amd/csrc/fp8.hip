// fp8.hip -- rows to e4m3 with a scale per 128 columns (moe_fp8_quant), FP8
// weight packing, and the product with block scales (moe_fp8_gemm,
// moe_fp8_proj).
#include "fp8_dev.h"
#include "fp8_launch.h"
#include "fp8_tile.h"
#include "host.h"

namespace moeblk {
namespace {

// ---------------------------------------------------------------- quantise
//
// A (row, 128-column block) is 8 lanes of 16 columns: its magnitude maximum is
// three butterfly steps, each lane stores 16 bytes. Division by the scale is an
// exact multiplication (a power of two), so the only rounding is e4m3's.
template <typename T, bool kVec>
__device__ __forceinline__ void load16(const T* row, int c0, int K, float v[16]) {
  if constexpr (kVec) {
    if (c0 + 16 <= K) {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const u32x4_t w = *reinterpret_cast<const u32x4_t*>(row + c0 + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = bf16_lo(w[j]);
            v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t w = *reinterpret_cast<const f32x4_t*>(row + c0 + 4 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float f = 0.0f;
    if (c0 + i < K) {
      if constexpr (sizeof(T) == 2)
        f = bf16_to_f32(row[c0 + i]);
      else
        f = row[c0 + i];
    }
    v[i] = f;
  }
}

// nrows: rows to quantise, or NULL for all `M` (a device count, for bucket rows)
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void quant_kernel(const T* __restrict__ x,
                                                    uint8_t* __restrict__ xq,
                                                    float* __restrict__ xs, int M, int K, int Kb,
                                                    const int32_t* __restrict__ nrows) {
  const size_t item = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int l8 = threadIdx.x & 7;
  const size_t row = item / Kb;
  const int kb = static_cast<int>(item - row * Kb);
  const int n = nrows ? min(*nrows, M) : M;
  if (row >= static_cast<size_t>(n)) return;
  float v[16];
  load16<T, kVec>(x + row * K, kb * kFp8Block + l8 * 16, K, v);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max_mag(m, v[i]);
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) m = max_mag(m, __shfl_xor(m, s, kWave));
  float inv;
  const float sc = fp8_block_scale(m, inv);
  u32x4_t q;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = pack_e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  *reinterpret_cast<u32x4_t*>(xq + row * (static_cast<size_t>(Kb) * kFp8Block) + kb * kFp8Block +
                              l8 * 16) = q;
  if (l8 == 0) xs[static_cast<size_t>(kb) * M + row] = sc;
}

// ---------------------------------------------------------------- packing

// one thread 16 bytes of the packed matrix; gate_up: rows in packed_row's
// interleaved order (common.h), else in order
__global__ __launch_bounds__(256) void pack_fp8_kernel(const uint8_t* __restrict__ q,
                                                       const float* __restrict__ sc,
                                                       uint8_t* __restrict__ out, int N, int K,
                                                       int Kb, int which, size_t pieces,
                                                       size_t packed_bytes) {
  const size_t p = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  const uint8_t* qm = q + static_cast<size_t>(blockIdx.y) * N * K;
  uint8_t* om = out + blockIdx.y * packed_bytes;
  if (p < pieces) {
    const size_t tile = p >> 7;
    const int h = static_cast<int>(p >> 6) & 1, lane = static_cast<int>(p) & 63;
    const int kb = static_cast<int>(tile % Kb);
    const int rt = static_cast<int>(tile / Kb);
    const int n = packed_row(which, N / 2, rt >> 2, rt & 3, lane & 15);
    const int k0 = kb * kFp8Block + 32 * (lane >> 4) + 16 * h;
    u32x4_t v = {0, 0, 0, 0};
    if (n < N) {
      const uint8_t* src = qm + static_cast<size_t>(n) * K + k0;
      if (k0 + 16 <= K && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        v = *reinterpret_cast<const u32x4_t*>(src);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (k0 + i < K) v[i >> 2] |= static_cast<uint32_t>(src[i]) << (8 * (i & 3));
      }
    }
    *reinterpret_cast<u32x4_t*>(om + p * 16) = v;
  }
  const size_t ns = static_cast<size_t>((N + 127) / 128) * Kb;
  if (p < ns)
    reinterpret_cast<float*>(om + pieces * 16)[p] = sc[blockIdx.y * ns + p];
}

// ---------------------------------------------------------------- product

__device__ __forceinline__ void store_out(void* out, size_t at, float v, bool bf16) {
  if (bf16)
    reinterpret_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(f32_to_bf16_bits(v));
  else
    reinterpret_cast<float*>(out)[at] = v;
}

// One workgroup: 16 kRT weight rows x 16 kTT tokens, its 8 waves taking every
// eighth K block. Each 128-K block is summed from zero (exact form, fp8_dev.h), scaled
// in fp32 by (token scale x weight scale) into the running sum; the waves' sums
// are added in wave order (deterministic).
template <int kRT, int kTT>
__global__ __launch_bounds__(512) void gemm_kernel(const uint8_t* __restrict__ xq,
                                                   const float* __restrict__ xs,
                                                   const uint8_t* __restrict__ w,
                                                   const float* __restrict__ ws,
                                                   void* __restrict__ out, int M, int N, int Kb,
                                                   bool out_bf16, int row_blocks) {
  __shared__ f32x4_t red[8][kRT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int rb = blockIdx.x % row_blocks, tg = blockIdx.x / row_blocks;
  const size_t Kp = static_cast<size_t>(Kb) * kFp8Block;
  const uint8_t* wt = w + static_cast<size_t>(rb) * kRT * Kb * kFp8TileBytes + lane * 16;
  const float* wsr = ws + static_cast<size_t>(rb * 16 * kRT / 128) * Kb;
  int tok[kTT];
  f32x4_t acc[kRT][kTT];
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    tok[t] = min((tg * kTT + t) * 16 + m16, M - 1);
#pragma unroll
    for (int r = 0; r < kRT; ++r) acc[r][t] = f32x4_t{0, 0, 0, 0};
  }
  for (int kb = wave; kb < Kb; kb += 8) {
    Bf16Frag a[kRT];
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      const uint8_t* p = wt + (static_cast<size_t>(r) * Kb + kb) * kFp8TileBytes;
      a[r] = e4m3_to_bf16(join8(ld_nt<u32x4_t>(p), ld_nt<u32x4_t>(p + 1024)));
    }
    const float sw = wsr[kb];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const uint8_t* p = xq + tok[t] * Kp + kb * kFp8Block + 32 * g;
      const Bf16Frag b = e4m3_to_bf16(join8(*reinterpret_cast<const u32x4_t*>(p),
                                            *reinterpret_cast<const u32x4_t*>(p + 16)));
      const float s = xs[static_cast<size_t>(kb) * M + tok[t]] * sw;
#pragma unroll
      for (int r = 0; r < kRT; ++r) {
        const f32x4_t d = mfma_exact_block(a[r], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(d[i], s, acc[r][t][i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRT; ++r) red[wave][r][lane] = acc[r][t];
    __syncthreads();
    if (wave < kRT) {
      f32x4_t s = red[0][wave][lane];
#pragma unroll
      for (int v = 1; v < 8; ++v) s += red[v][wave][lane];
      const int token = (tg * kTT + t) * 16 + m16;
      const int n0 = (rb * kRT + wave) * 16 + 4 * g;
      if (token < M) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < N) store_out(out, static_cast<size_t>(token) * N + n0 + i, s[i], out_bf16);
      }
    }
  }
}

}  // namespace

void launch_fp8_quant(const void* x, int in_type, uint8_t* xq, float* xs, int M, int K,
                      const int32_t* nrows, hipStream_t stream) {
  const int Kb = fp8_kb(K);
  const dim3 grid(static_cast<unsigned>((static_cast<size_t>(M) * Kb * 8 + 255) / 256));
  if (in_type == MOE_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(x);
    if (K % 8 == 0)
      quant_kernel<uint16_t, true><<<grid, 256, 0, stream>>>(p, xq, xs, M, K, Kb, nrows);
    else
      quant_kernel<uint16_t, false><<<grid, 256, 0, stream>>>(p, xq, xs, M, K, Kb, nrows);
  } else {
    const float* p = static_cast<const float*>(x);
    if (K % 4 == 0)
      quant_kernel<float, true><<<grid, 256, 0, stream>>>(p, xq, xs, M, K, Kb, nrows);
    else
      quant_kernel<float, false><<<grid, 256, 0, stream>>>(p, xq, xs, M, K, Kb, nrows);
  }
}

void launch_fp8_pack(const void* q, const void* scales, void* packed, int n, int N, int K,
                     int which, hipStream_t stream) {
  const int Kb = fp8_kb(K);
  const size_t pieces = fp8_tile_bytes(N, K) / 16;
  const dim3 grid(static_cast<unsigned>((pieces + 255) / 256), n);
  pack_fp8_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint8_t*>(q),
                                            static_cast<const float*>(scales),
                                            static_cast<uint8_t*>(packed), N, K, Kb, which, pieces,
                                            fp8_packed_bytes(N, K));
}

namespace {

template <int kRT, int kTT, int kWN, int kWM, bool kExact>
void launch_tiles(Fp8TileArgs a, hipStream_t stream) {
  constexpr int BN = 16 * kRT * kWN, BM = 16 * kTT * kWM;
  a.tiles_n = (a.N + BN - 1) / BN;
  a.tiles_m = (a.M + BM - 1) / BM;
  const unsigned grid = static_cast<unsigned>(a.tiles_n) * a.tiles_m;
  fp8_tile_kernel<kRT, kTT, kWN, kWM, kExact><<<grid, 64 * kWN * kWM, 0, stream>>>(a);
}

void launch_fp8_gemm(const moe_fp8_dims& m, const void* xq, const float* xs, const void* packed,
                     void* out, hipStream_t stream) {
  const int Kb = fp8_kb(m.K);
  const uint8_t* q = static_cast<const uint8_t*>(xq);
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  const float* ws = reinterpret_cast<const float*>(w + fp8_tile_bytes(m.N, m.K));
  const bool bf = m.out_type == MOE_BF16;
  if (m.M > 128) {
    const Fp8TileArgs a = {q, xs, w, ws, out, m.M, m.N, Kb, bf, 0, 0};
    // A step of one 256 x 256 tile a CU takes about 2.1 us, of two 128 x 128
    // tiles 1.25 us; rounds over the 256 CUs times that decide. Measured (us,
    // K = 7168, N = 4096, 256 against 128 tiles): M = 8192 240 / 259, M = 4096
    // 122 / 135, M = 2048 107 / 69.5.
    const auto rounds = [&](int tile, int slots) {
      const size_t t = static_cast<size_t>((m.N + tile - 1) / tile) * ((m.M + tile - 1) / tile);
      return (t + slots - 1) / slots;
    };
    if (!bf)
      launch_tiles<4, 4, 2, 2, true>(a, stream);
    else if (rounds(256, 256) * 210 <= rounds(128, 512) * 125)
      launch_tiles<8, 4, 2, 4, false>(a, stream);
    else
      launch_tiles<4, 4, 2, 2, false>(a, stream);
    return;
  }
  const int rbs = (m.N + 63) / 64;
  const int tgs = m.M <= 16 ? 1 : (m.M + 63) / 64;
  const dim3 grid(static_cast<unsigned>(rbs) * tgs);
  if (m.M <= 16)
    gemm_kernel<4, 1><<<grid, 512, 0, stream>>>(q, xs, w, ws, out, m.M, m.N, Kb, bf, rbs);
  else
    gemm_kernel<4, 4><<<grid, 512, 0, stream>>>(q, xs, w, ws, out, m.M, m.N, Kb, bf, rbs);
}

size_t gemm_workspace(const moe_fp8_dims&) { return 256; }
size_t quant_bytes(const moe_fp8_dims& m) {
  return round_up(static_cast<size_t>(m.M) * fp8_kb(m.K) * kFp8Block, 256);
}
size_t quant_scale_bytes(const moe_fp8_dims& m) {
  return round_up(static_cast<size_t>(m.M) * fp8_kb(m.K) * 4, 256);
}

}  // namespace
}  // namespace moeblk

using namespace moeblk;

extern "C" {

int moe_check_fp8_dims(const moe_fp8_dims* dims) { return check_fp8_dims(dims); }

size_t moe_packed_fp8_bytes(const moe_fp8_dims* dims) {
  return check_fp8_dims(dims) ? 0 : fp8_packed_bytes(dims->N, dims->K);
}

int moe_pack_fp8(const moe_fp8_dims* dims, const void* q, const float* scales, void* packed,
                 hipStream_t stream) {
  const int rc = check_fp8_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(q && scales && packed, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(q) && aligned16(scales) && aligned16(packed), MOE_ERR_ALIGN);
  launch_fp8_pack(q, scales, packed, 1, dims->N, dims->K, MOE_W2, stream);
  return launch_status();
}

int moe_fp8_quant(const moe_fp8_dims* dims, const void* x, void* xq, float* xs,
                  hipStream_t stream) {
  const int rc = check_fp8_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(x && xq && xs, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(x) && aligned16(xq) && aligned16(xs), MOE_ERR_ALIGN);
  launch_fp8_quant(x, dims->in_type, static_cast<uint8_t*>(xq), xs, dims->M, dims->K, nullptr,
                   stream);
  return launch_status();
}

size_t moe_fp8_gemm_workspace_bytes(const moe_fp8_dims* dims) {
  return check_fp8_dims(dims) ? 0 : gemm_workspace(*dims);
}

int moe_fp8_gemm(const moe_fp8_dims* dims, const void* xq, const float* xs, const void* w_packed,
                 void* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_fp8_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(xq && xs && w_packed && out && workspace, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(xq) && aligned16(xs) && aligned16(w_packed) && aligned16(out) &&
                  aligned16(workspace),
              MOE_ERR_ALIGN);
  MOE_REQUIRE(workspace_bytes >= gemm_workspace(*dims), MOE_ERR_WORKSPACE);
  launch_fp8_gemm(*dims, xq, xs, w_packed, out, stream);
  return launch_status();
}

size_t moe_fp8_proj_workspace_bytes(const moe_fp8_dims* dims) {
  return check_fp8_dims(dims) ? 0
                              : gemm_workspace(*dims) + quant_bytes(*dims) +
                                    quant_scale_bytes(*dims);
}

int moe_fp8_proj(const moe_fp8_dims* dims, const void* x, const void* w_packed, void* out,
                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_fp8_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(x && w_packed && out && workspace, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(x) && aligned16(w_packed) && aligned16(out) && aligned16(workspace),
              MOE_ERR_ALIGN);
  MOE_REQUIRE(workspace_bytes >= moe_fp8_proj_workspace_bytes(dims), MOE_ERR_WORKSPACE);
  uint8_t* xq = static_cast<uint8_t*>(workspace) + gemm_workspace(*dims);
  float* xs = reinterpret_cast<float*>(xq + quant_bytes(*dims));
  launch_fp8_quant(x, dims->in_type, xq, xs, dims->M, dims->K, nullptr, stream);
  launch_fp8_gemm(*dims, xq, xs, w_packed, out, stream);
  return launch_status();
}

}  // extern "C"
