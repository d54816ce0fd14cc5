// fp8.hip -- rows to e4m3 with a scale per 128 columns (moe_fp8_quant), FP8
// weight packing, and the product with block scales (moe_fp8_gemm,
// moe_fp8_proj).
#include <type_traits>

#include "fp8_dev.h"
#include "fp8_launch.h"
#include "fp8_quant.h"
#include "fp8_tile.h"
#include "host.h"

namespace moeblk {
namespace {

// ---------------------------------------------------------------- quantise
//
// One pass over the rows, bound by memory: 16384 x 7168 bf16 in 63.5 us, 5.6 TB/s.

template <typename T>
__global__ __launch_bounds__(256) void quant_kernel(const T* __restrict__ x,
                                                    uint8_t* __restrict__ xq,
                                                    float* __restrict__ xs, int M, int K, int Kb) {
  const size_t item = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int l8 = threadIdx.x & 7;
  const size_t row = item / Kb;
  const int kb = static_cast<int>(item - row * Kb);
  if (row >= static_cast<size_t>(M)) return;
  Raw16<T> v;
  float sc;
  load16<T>(x + row * K, kb * kFp8Block + l8 * 16, K, v);
  const u32x4_t q = quant16(v, sc);
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

// ---------------------------------------------------------------- product, few rows
//
// At most 16 rows: the weight is read once and its bytes bound the call. A
// workgroup takes 16 kRT weight rows; its kNW waves take every kNW-th K block, a
// ring of kRing blocks' loads in flight each, straight from the packed order into
// registers (exact form, fp8_dev.h). The waves' sums are added in wave order.
//
// kSrc says where the rows come from. kRowsX: the rows themselves; every
// workgroup quantises them into LDS while its first weight loads are in flight,
// which costs less than a launch in front as long as they are few (rows x K
// blocks up to kFusedItems): 1 x 4096 x 7168 15.6 us a call with the launch, 7.6 without
// (29 MB of weights, 3.9 TB/s). kRowsQ: quantised rows, read from memory.
enum RowSource { kRowsBf16, kRowsFp32, kRowsQ };

constexpr int kFusedItems = 896;  // most (row, K block) pairs in LDS, 132 bytes each
constexpr int kFewItems = 256;    // few enough for several workgroups a CU

struct RowsArgs {
  const void* x;      // kRowsBf16, kRowsFp32: [M][K]
  const uint8_t* xq;  // kRowsQ
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  int M, N, K, Kb;
  bool out_bf16;
  int row_blocks;
  SplitK split;
};

template <int kRT, int kNW, int kSrc, int kItems>
__global__ __launch_bounds__(64 * kNW) void rows_kernel(RowsArgs a) {
  constexpr int kRing = kRT == 1 ? 4 : 2;
  constexpr bool kFused = kSrc != kRowsQ;
  __shared__ f32x4_t red[kNW][kRT][64];
  __shared__ __attribute__((aligned(128))) uint8_t xl[kFused ? kItems * kFp8Block : 16];
  __shared__ float sl[kFused ? kItems : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int Kb = a.Kb, M = a.M;
  const int rb = blockIdx.x % a.row_blocks, part = blockIdx.x / a.row_blocks;
  int kb0, kb1;
  part_range(Kb, a.split.parts, part, kb0, kb1);
  const uint8_t* wt = a.w + static_cast<size_t>(rb) * kRT * Kb * kFp8TileBytes + lane * 16;
  const float* wsr = a.ws + static_cast<size_t>(rb * 16 * kRT / 128) * Kb;
  const int tok = min(m16, M - 1);
  const uint8_t* xrow = kFused ? nullptr : a.xq + tok * (static_cast<size_t>(Kb) * kFp8Block) + 32 * g;

  u32x4_t wreg[kRing][kRT][2], xreg[kFused ? 1 : kRing][2];
  float sreg[kRing];
  const auto load = [&](int i, int kb) {
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      const uint8_t* p = wt + (static_cast<size_t>(r) * Kb + kb) * kFp8TileBytes;
      wreg[i][r][0] = ld_nt<u32x4_t>(p);
      wreg[i][r][1] = ld_nt<u32x4_t>(p + 1024);
    }
    sreg[i] = wsr[kb];
    if constexpr (!kFused) {
      sreg[i] *= a.xs[static_cast<size_t>(kb) * M + tok];
      xreg[i][0] = *reinterpret_cast<const u32x4_t*>(xrow + kb * kFp8Block);
      xreg[i][1] = *reinterpret_cast<const u32x4_t*>(xrow + kb * kFp8Block + 16);
    }
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i)
    if (kb0 + wave + kNW * i < kb1) load(i, kb0 + wave + kNW * i);

  if constexpr (kFused) {
    // item (kb - kb0) * M + row: 8 lanes of 16 columns; the 16-byte chunks of a
    // row permuted by chunk ^ (row % 8)
    using T = typename std::conditional<kSrc == kRowsBf16, uint16_t, float>::type;
    const T* x = static_cast<const T*>(a.x);
    const int l8 = threadIdx.x & 7;
    for (int item = threadIdx.x >> 3; item < M * (kb1 - kb0); item += 8 * kNW) {
      const int row = item % M, kb = kb0 + item / M;
      Raw16<T> v;
      load16<T>(x + static_cast<size_t>(row) * a.K, kb * kFp8Block + l8 * 16, a.K, v);
      float sc;
      const u32x4_t q = quant16(v, sc);
      *reinterpret_cast<u32x4_t*>(xl + item * kFp8Block + ((l8 ^ (row & 7)) * 16)) = q;
      if (l8 == 0) sl[item] = sc;
    }
    __syncthreads();
  }

  f32x4_t acc[kRT];
#pragma unroll
  for (int r = 0; r < kRT; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
  const int c0 = ((2 * g) ^ (tok & 7)) * 16, c1 = ((2 * g + 1) ^ (tok & 7)) * 16;
  for (int base = kb0 + wave; base < kb1; base += kNW * kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      const int kb = base + kNW * i;
      if (kb < kb1) {
        Bf16Frag b;
        float s = sreg[i];
        if constexpr (kFused) {
          const int item = (kb - kb0) * M + tok;
          const uint8_t* p = xl + item * kFp8Block;
          b = e4m3_to_bf16(join8(*reinterpret_cast<const u32x4_t*>(p + c0),
                                 *reinterpret_cast<const u32x4_t*>(p + c1)));
          s *= sl[item];
        } else {
          b = e4m3_to_bf16(join8(xreg[i][0], xreg[i][1]));
        }
#pragma unroll
        for (int r = 0; r < kRT; ++r) {
          const f32x4_t d = mfma_exact_block(e4m3_to_bf16(join8(wreg[i][r][0], wreg[i][r][1])), b);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[r][c] = __builtin_fmaf(d[c], s, acc[r][c]);
        }
        if (kb + kNW * kRing < kb1) load(i, kb + kNW * kRing);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRT; ++r) red[wave][r][lane] = acc[r];
  __syncthreads();
  f32x4_t sum[1] = {{0, 0, 0, 0}};
  if (wave < kRT) {
    sum[0] = red[0][wave][lane];
#pragma unroll
    for (int v = 1; v < kNW; ++v) sum[0] += red[v][wave][lane];
  }
  __shared__ int last;
  if (!join_parts(a.split, rb, part, wave < kRT, sum, &last)) return;
  if (wave < kRT && m16 < M) {
    const int n0 = (rb * kRT + wave) * 16 + 4 * g;
    store4<true>(a.out, static_cast<size_t>(m16) * a.N + n0, a.N - n0, sum[0],
                 a.out_bf16);
  }
}

// ---------------------------------------------------------------- product, from 17 rows
//
// 16 kRT weight rows x 16 kTT tokens a workgroup; its 8 waves take every eighth K
// block of the workgroup's part, one or two blocks' loads in flight (kRing),
// straight into registers (tokens through L2). The waves' sums are added through
// LDS, all threads taking part. 128 x 7168 x 2048: 11.7 us (one 8-wave workgroup a CU,
// one K block's loads in flight a wave).
struct MidArgs {
  const uint8_t* xq;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  int M, N, Kb;
  bool out_bf16;
  int row_blocks, tiles;
  SplitK split;
};

__device__ __forceinline__ u32x4_t buffer16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

template <int kRT, int kTT, bool kExact, int kRing>
__device__ __forceinline__ void mid_body(const MidArgs& a, f32x4_t* red, int* last) {
  constexpr int kEach = (kRT * kTT + 7) / 8;  // tiles a wave adds up at the end
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  const int part = blockIdx.x / a.tiles, tile = blockIdx.x - part * a.tiles;
  const int rb = tile % a.row_blocks, t0 = tile / a.row_blocks * 16 * kTT;
  const int Kb = a.Kb, M = a.M;
  int kb0, kb1;
  part_range(Kb, a.split.parts, part, kb0, kb1);
  const uint32_t Kp = static_cast<uint32_t>(Kb) * kFp8Block;
  const auto rsrc = [](const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes),
                                             0x00020000);
  };
  const __amdgpu_buffer_rsrc_t wr =
      rsrc(a.w + static_cast<size_t>(rb) * kRT * Kb * kFp8TileBytes, kRT * Kb * kFp8TileBytes);
  const __amdgpu_buffer_rsrc_t xr = rsrc(a.xq, M * Kp), sr = rsrc(a.xs, M * Kb * 4);
  const float* wsr = a.ws + static_cast<size_t>(rb * kRT / 8) * Kb;
  uint32_t tok[kTT];
  f32x4_t acc[kRT][kTT];
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    tok[t] = min(t0 + t * 16 + m16, M - 1);
#pragma unroll
    for (int r = 0; r < kRT; ++r) acc[r][t] = f32x4_t{0, 0, 0, 0};
  }
  u32x4_t w[kRing][kRT][2], x[kRing][kTT][2];
  float s[kRing][kTT], sw[kRing];
  const auto load = [&](int i, int kb) {
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      const uint32_t at = static_cast<uint32_t>(r * Kb + kb) * kFp8TileBytes;
      w[i][r][0] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16, at, kCpolNt));
      w[i][r][1] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16, at + 1024, kCpolNt));
    }
    sw[i] = wsr[kb];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const uint32_t v = tok[t] * Kp + 32 * g;
      x[i][t][0] = buffer16(xr, v, kb * kFp8Block);
      x[i][t][1] = buffer16(xr, v + 16, kb * kFp8Block);
      s[i][t] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(sr, tok[t] * 4, kb * M * 4, 0));
    }
  };
  const auto multiply = [&](int i) {
    Bf16Frag xe[kExact ? kTT : 1];
    float f[kTT];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      f[t] = s[i][t] * sw[i];
      if constexpr (kExact) xe[t] = e4m3_to_bf16(join8(x[i][t][0], x[i][t][1]));
    }
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
      const i32x8_t w8 = join8(w[i][r][0], w[i][r][1]);
      Bf16Frag we;
      if constexpr (kExact) we = e4m3_to_bf16(w8);
#pragma unroll
      for (int t = 0; t < kTT; ++t) {
        f32x4_t d;
        if constexpr (kExact)
          d = mfma_exact_block(we, xe[t]);
        else
          d = mfma_fp8_block(w8, join8(x[i][t][0], x[i][t][1]));
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][t][c] = __builtin_fmaf(d[c], f[t], acc[r][t][c]);
      }
    }
  };
  if constexpr (kRing == 2) {
    int kb = kb0 + uwave;
    if (kb < kb1) load(0, kb);
    if (kb + 8 < kb1) load(1, kb + 8);
    for (; kb < kb1; kb += 16) {
      multiply(0);
      if (kb + 16 < kb1) load(0, kb + 16);
      if (kb + 8 < kb1) {
        multiply(1);
        if (kb + 24 < kb1) load(1, kb + 24);
      }
    }
  } else {
    for (int kb = kb0 + uwave; kb < kb1; kb += 8) {
      load(0, kb);
      multiply(0);
    }
  }
  // rounds of 8 tiles (tile i = r kTT + t), a tile a wave: red[wave][8][lane]
  f32x4_t sum[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (e) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8 && e * 8 + i < kRT * kTT; ++i)
      red[(wave * 8 + i) * 64 + lane] = acc[(e * 8 + i) / kTT][(e * 8 + i) % kTT];
    __syncthreads();
    sum[e] = red[wave * 64 + lane];
#pragma unroll
    for (int v = 1; v < 8; ++v) sum[e] += red[(v * 8 + wave) * 64 + lane];
  }
  if (!join_parts(a.split, tile, part, true, sum, last)) return;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * 8 + wave, token = t0 + (i % kTT) * 16 + m16;
    const int n0 = (rb * kRT + i / kTT) * 16 + 4 * g;
    if (token < M && i < kRT * kTT)
      store4<kExact>(a.out, static_cast<size_t>(token) * a.N + n0, a.N - n0, sum[e], a.out_bf16);
  }
}

template <int kRT, int kTT, bool kExact, int kRing>
__global__ __launch_bounds__(512) void mid_kernel(MidArgs a) {
  __shared__ f32x4_t red[8 * 8 * 64];
  __shared__ int last;
  mid_body<kRT, kTT, kExact, kRing>(a, red, &last);
}

}  // namespace

void launch_fp8_quant(const void* x, int in_type, uint8_t* xq, float* xs, int M, int K,
                      hipStream_t stream) {
  const int Kb = fp8_kb(K);
  const dim3 grid(static_cast<unsigned>((static_cast<size_t>(M) * Kb * 8 + 255) / 256));
  if (in_type == MOE_BF16)
    quant_kernel<uint16_t><<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x), xq, xs, M, K, Kb);
  else
    quant_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), xq, xs, M, K, Kb);
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

// How a product of these sizes runs: the kernel, and its K parts: as many as
// bring the workgroups to the number of CUs, each with at least `least` K blocks
// (adding up P parts costs the last workgroup of a tile about 2 us). Measured, us,
// split / whole: M = 8, N = 512, K = 8192 6.0 / 9.3; M = 64, N = 4096, K = 7168
// 18.0 / 21.9; M = 512, N = 4096, K = 7168 43 / 57.
enum Form { kRows, kMid, kTile128, kTile256 };
struct Plan {
  Form form;
  int tiles, parts;
  size_t part_bytes;  // fp32 sums of one part of one tile
};

int split_parts(int tiles, int Kb, int least) {
  if (tiles > kSplitTiles) return 1;
  int p = 256 / tiles;
  p = p < Kb / least ? p : Kb / least;
  return p < 1 ? 1 : p;
}

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// few rows: 16 weight rows a workgroup while that gives at most 512 workgroups, else 64
inline bool thin_rows(int N) { return N <= 16 * 512; }
// From 17 rows: 32 tokens a workgroup while they are all, else 64; 32 weight rows
// while that gives no more workgroups than CUs, else 64 (half the token bytes
// through L2, but only one K block's loads at a time fit the registers at 64
// tokens). Measured, us with the quantisation, 32 / 64 rows: M = 128, N = 7168, K
// = 2048 18.2 / 13.3; M = 128, N = 512, K = 8192 12.0 / 15.0; M = 64, N = 4096, K =
// 7168 18.0 / 18.6; M = 77, N = 4099, K = 2120 (258 / 130 workgroups) 15.3 / 15.2.
inline int mid_tiles_m(const moe_fp8_dims& m) { return ceil_div(m.M, m.M <= 32 ? 32 : 64); }
inline int mid_rows(const moe_fp8_dims& m) {
  return ceil_div(m.N, 32) * mid_tiles_m(m) <= 256 ? 32 : 64;
}

// The register kernel (mid) or LDS tiles: mid for one 64-token group, and while its
// 64-row tiles are few; with more, the tokens' bytes through L2 cost more than
// the tiles' steps. Measured, us with the quantisation, mid / tiles: M = 160, N =
// 1000, K = 1000 7.6 / 12.5; M = 160, N = 4096, K = 7168 27.5 / 32.4; M = 300, N = 4096,
// K = 4096 30.2 / 29.6; M = 128, N = 16384, K = 4096 35.9 / 33.8; M = 512, N = 4096, K =
// 7168 51.7 / 42.9.
inline bool use_mid(const moe_fp8_dims& m) {
  return m.M <= 64 || ceil_div(m.N, 64) * ceil_div(m.M, 64) <= 320;
}

// The exact form of the block sums (fp8_dev.h): always for fp32 outputs, at M <= 16, and
// in the register kernel up to 128 rows (a decode step's), which loads bound. Measured, us
// with the quantisation, fast / exact: M = 32, N = 4096, K = 7168 13.8 / 14.3; M = 64 17.2
// / 18.2; M = 128, N = 7168, K = 2048 12.7 / 13.3. Beyond, the matrix rate counts: M = 160,
// N = 4096, K = 7168 27.5 / 32.0; M = 300, K = 4096 30.1 / 35.7; in LDS tiles M = 1024, K =
// 7168 58 / 71, M = 2048 76 / 116.
inline bool exact_sums(const moe_fp8_dims& m) {
  return m.out_type == MOE_FP32 || (m.M <= 128 && use_mid(m));
}

Plan fp8_plan(const moe_fp8_dims& m) {
  const int Kb = fp8_kb(m.K);
  Plan p;
  if (m.M <= 16) {
    p.form = kRows;
    p.tiles = thin_rows(m.N) ? ceil_div(m.N, 16) : ceil_div(m.N, 64);
    p.parts = split_parts(p.tiles, Kb, 16);
    p.part_bytes = 1024 * 16;
    return p;
  }
  if (use_mid(m)) {
    p.form = kMid;
    p.tiles = ceil_div(m.N, mid_rows(m)) * mid_tiles_m(m);
    p.parts = split_parts(p.tiles, Kb, 8);
    p.part_bytes = 2 * 512 * 16;
    return p;
  }
  // A step of one 256 x 256 tile a CU takes about 1.9 us, of two 128 x 128
  // tiles 1.25 us; rounds over the 256 CUs times that decide. Measured (us,
  // K = 7168, N = 4096, 256 against 128 tiles): M = 8192 210 / 259, M = 4096
  // 109 / 135, M = 2048 104 / 69.5.
  const auto rounds = [&](int tile, int slots) {
    const size_t t = static_cast<size_t>(ceil_div(m.N, tile)) * ceil_div(m.M, tile);
    return (t + slots - 1) / slots;
  };
  if (m.out_type == MOE_BF16 && rounds(256, 256) * 190 <= rounds(128, 512) * 125) {
    p.form = kTile256;
    p.tiles = ceil_div(m.N, 256) * ceil_div(m.M, 256);
    p.parts = 1;
  } else {
    p.form = kTile128;
    p.tiles = ceil_div(m.N, 128) * ceil_div(m.M, 128);
    p.parts = split_parts(p.tiles, Kb, 8);
  }
  p.part_bytes = 16 * 256 * 16;
  return p;
}

size_t gemm_workspace(const moe_fp8_dims& m) {
  const Plan p = fp8_plan(m);
  return kSplitCounterBytes + (p.parts > 1 ? p.tiles * p.parts * p.part_bytes : 0);
}

SplitK split_of(const Plan& p, void* workspace) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return SplitK{p.parts, reinterpret_cast<int32_t*>(ws),
                reinterpret_cast<f32x4_t*>(ws + kSplitCounterBytes)};
}

template <int kRT, int kTT, int kWN, int kWM, bool kExact>
void launch_tiles(Fp8TileArgs a, hipStream_t stream) {
  a.tiles_n = ceil_div(a.N, 16 * kRT * kWN);
  a.tiles_m = ceil_div(a.M, 16 * kTT * kWM);
  const unsigned grid = static_cast<unsigned>(a.tiles_n) * a.tiles_m * a.split.parts;
  fp8_tile_kernel<kRT, kTT, kWN, kWM, kExact><<<grid, 64 * kWN * kWM, 0, stream>>>(a);
}

// 16 waves where a workgroup has a CU to itself and 8 could not have all of its K
// blocks in flight. Measured, us, 16 / 8 waves: N = 4096, K = 7168, M = 16 13.3 /
// 16.5; N = 4096, K = 4096, M = 8 7.3 / 7.6; N = 7168, K = 2048, M = 1 7.3 / 5.8;
// N = 1024, K = 4096, M = 8 7.1 / 6.7.
template <int kSrc>
void launch_rows(RowsArgs a, const Plan& p, hipStream_t stream) {
  const int Kpart = ceil_div(a.Kb, p.parts);
  const unsigned grid = p.tiles * p.parts;
  a.row_blocks = p.tiles;
  const auto launch = [&](auto items) {
    constexpr int kItems = decltype(items)::value;
    if (!thin_rows(a.N))
      rows_kernel<4, 8, kSrc, kItems><<<grid, 512, 0, stream>>>(a);
    else if (grid <= 256 && Kpart > 32)
      rows_kernel<1, 16, kSrc, kItems><<<grid, 1024, 0, stream>>>(a);
    else
      rows_kernel<1, 8, kSrc, kItems><<<grid, 512, 0, stream>>>(a);
  };
  if constexpr (kSrc == kRowsQ)
    launch(std::integral_constant<int, 0>());
  else if (a.M * Kpart <= kFewItems)
    launch(std::integral_constant<int, kFewItems>());
  else
    launch(std::integral_constant<int, kFusedItems>());
}

void launch_mid(const MidArgs& a, int rows, bool exact, unsigned grid, hipStream_t stream) {
  const auto launch = [&](auto kernel) { kernel<<<grid, 512, 0, stream>>>(a); };
  const bool small = rows == 32;
  if (a.M <= 32)
    small ? launch(mid_kernel<2, 2, true, 2>) : launch(mid_kernel<4, 2, true, 1>);
  else if (exact)
    small ? launch(mid_kernel<2, 4, true, 2>) : launch(mid_kernel<4, 4, true, 1>);
  else
    small ? launch(mid_kernel<2, 4, false, 2>) : launch(mid_kernel<4, 4, false, 1>);
}

void launch_fp8_gemm(const moe_fp8_dims& m, const void* xq, const float* xs, const void* packed,
                     void* out, void* workspace, hipStream_t stream) {
  const int Kb = fp8_kb(m.K);
  const uint8_t* q = static_cast<const uint8_t*>(xq);
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  const float* ws = reinterpret_cast<const float*>(w + fp8_tile_bytes(m.N, m.K));
  const bool bf = m.out_type == MOE_BF16;
  const Plan p = fp8_plan(m);
  const SplitK split = split_of(p, workspace);
  if (p.form == kRows) {
    launch_rows<kRowsQ>(RowsArgs{nullptr, q, xs, w, ws, out, m.M, m.N, m.K, Kb, bf, 0, split}, p,
                        stream);
  } else if (p.form == kMid) {
    const MidArgs a = {q, xs, w, ws, out, m.M, m.N, Kb, bf, ceil_div(m.N, mid_rows(m)), p.tiles, split};
    launch_mid(a, mid_rows(m), exact_sums(m), p.tiles * p.parts, stream);
  } else {
    const Fp8TileArgs a = {q, xs, w, ws, out, m.M, m.N, Kb, bf, 0, 0, split};
    if (p.form == kTile256)
      launch_tiles<8, 4, 2, 4, false>(a, stream);
    else if (bf)
      launch_tiles<4, 4, 2, 2, false>(a, stream);
    else
      launch_tiles<4, 4, 2, 2, true>(a, stream);
  }
}

// few rows, quantised by the product's own workgroups; false if that is not for them
bool launch_fp8_fused(const moe_fp8_dims& m, const void* x, const void* packed, void* out,
                      void* workspace, hipStream_t stream) {
  const Plan p = fp8_plan(m);
  const int Kb = fp8_kb(m.K);
  if (p.form != kRows || m.M * ceil_div(Kb, p.parts) > kFusedItems) return false;
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  const float* ws = reinterpret_cast<const float*>(w + fp8_tile_bytes(m.N, m.K));
  const RowsArgs a = {x,   nullptr, nullptr, w,  ws, out, m.M, m.N, m.K, Kb, m.out_type == MOE_BF16,
                      0, split_of(p, workspace)};
  if (m.in_type == MOE_BF16)
    launch_rows<kRowsBf16>(a, p, stream);
  else
    launch_rows<kRowsFp32>(a, p, stream);
  return true;
}

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
  launch_fp8_quant(x, dims->in_type, static_cast<uint8_t*>(xq), xs, dims->M, dims->K, stream);
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
  launch_fp8_gemm(*dims, xq, xs, w_packed, out, workspace, stream);
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
  if (!launch_fp8_fused(*dims, x, w_packed, out, workspace, stream)) {
    launch_fp8_quant(x, dims->in_type, xq, xs, dims->M, dims->K, stream);
    launch_fp8_gemm(*dims, xq, xs, w_packed, out, workspace, stream);
  }
  return launch_status();
}

}  // extern "C"
