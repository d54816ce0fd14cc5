// mx.hip -- rows to MXFP4 and back (moe_mx_quant, moe_mx_dequant), packing of a
// weight, and the product of such rows and a packed weight (moe_mx_gemm, moe_mx_proj).
#include <type_traits>

#include "fp8_quant.h"
#include "host.h"
#include "mx_dev.h"
#include "mx_rows.h"
#include "mx_tile.h"

namespace moeblk {
namespace {

// ---------------------------------------------------------------- quantise, read back
//
// One pass over the rows, bound by memory. Two lanes share a block: 16 columns each,
// one DPP step for the maximum, 8 bytes of codes a lane. 16384 rows of 7168: 49 to 51 us from
// bf16 and 95 from fp32 (6.0 and 5.6 TB/s); 8 x 4096 2.4 us.

template <typename T>
__global__ __launch_bounds__(256) void mx_quant_kernel(const T* __restrict__ x,
                                                       uint8_t* __restrict__ q,
                                                       uint8_t* __restrict__ s, int M, int K,
                                                       int Kc) {
  const size_t item = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  const int per_row = Kc * 8;  // items: halves of blocks
  const size_t row = item / per_row;
  const int i = static_cast<int>(item - row * per_row);
  if (row >= static_cast<size_t>(M)) return;  // both lanes of a block or none
  Raw16<T> v;
  load16<T>(x + row * K, i * 16, K, v);
  uint32_t m = 0;
  if constexpr (sizeof(T) == 2) {
    u16x2_t p = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, v.w[j] & 0x7fff7fffu));
    m = static_cast<uint32_t>(p[0] > p[1] ? p[0] : p[1]) << 16;
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t a = v.w[j] & 0x7fffffffu;
      m = m > a ? m : a;
    }
  }
  m = max_dpp<0xb1>(m);  // lane ^ 1
  const uint32_t byte = mx_scale_byte(m);
  const float sc = e8m0_scale(byte);
  u32x2_t c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(T) == 2) {
      c[h] = mx_codes_bf16(&v.w[4 * h], sc);
    } else {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v.w[8 * h + j]);
      c[h] = mx_codes(f, sc);
    }
    c[h] = mx_codes_or_zero(c[h], byte);
  }
  *reinterpret_cast<u32x2_t*>(q + row * (static_cast<size_t>(Kc) * 64) + i * 8) = c;
  if ((i & 1) == 0) s[row * (static_cast<size_t>(Kc) * 4) + (i >> 1)] = static_cast<uint8_t>(byte);
}

// 16 bytes of values a thread, stored past the caches: 16384 rows of 7168 in 42 us as bf16 (47
// right behind their quantisation) and 73 us as fp32 (7.1 and 7.3 TB/s); stores through them took
// 63 and 105.
template <typename T>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ s,
                                                         T* __restrict__ x, int M, int K, int Kc) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  constexpr int kN = 16 / sizeof(T);
  const size_t item = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  const int per_row = (K + kN - 1) / kN;
  const size_t row = item / per_row;
  const int c = static_cast<int>(item - row * per_row) * kN;
  if (row >= static_cast<size_t>(M)) return;
  const uint8_t* codes = q + row * (static_cast<size_t>(Kc) * 64) + c / 2;
  const float sc = e8m0_scale(s[row * (static_cast<size_t>(Kc) * 4) + c / kMxBlock]);
  T* o = x + row * K + c;
  u32x4_t v;
  if constexpr (sizeof(T) == 4) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(codes);
    const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 0);
    const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 1);
    v = __builtin_bit_cast(u32x4_t, f32x4_t{p0[0], p0[1], p1[0], p1[1]});
  } else {
    v = __builtin_bit_cast(u32x4_t, decode_fp4x8(*reinterpret_cast<const uint32_t*>(codes), sc));
  }
  if (c + kN <= K) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any_t*>(o));
  } else {
#pragma unroll
    for (int i = 0; i < kN - 1; ++i) {
      if (c + i >= K) continue;
      if constexpr (sizeof(T) == 4)
        o[i] = __uint_as_float(v[i]);
      else
        o[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// ---------------------------------------------------------------- packing

// one workgroup a tile; rows and columns past the end are zeros of scale 1
__global__ __launch_bounds__(256) void mx_pack_kernel(const uint8_t* __restrict__ q,
                                                      const uint8_t* __restrict__ s,
                                                      uint8_t* __restrict__ out, int N, int K,
                                                      int Kc) {
  const int tile = blockIdx.x, c = tile % Kc, rb = tile / Kc;
  const int r = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int n = packed_row(MOE_W2, 0, rb, r, lane & 15);
  const int k0 = kChunkK * c + kMxBlock * (lane >> 4), left = K - k0;
  u32x4_t v = {0, 0, 0, 0};
  uint8_t byte = 127;
  if (n < N && left > 0) {
    v = *reinterpret_cast<const u32x4_t*>(q + static_cast<size_t>(n) * Kc * 64 + k0 / 2);
    byte = s[static_cast<size_t>(n) * Kc * 4 + k0 / kMxBlock];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int in = left - 8 * i;  // columns of this word inside the row
      if (in < 8) v[i] &= in <= 0 ? 0u : (1u << (4 * in)) - 1u;
    }
  }
  uint8_t* t = out + static_cast<size_t>(tile) * kMxTileBytes;
  *reinterpret_cast<u32x4_t*>(t + r * 1024 + lane * 16) = v;
  t[4096 + lane * 4 + r] = byte;
}

// ---------------------------------------------------------------- product

struct MxGemmArgs {
  const void* x;  // rows as they are (K values each), or NULL
  const uint8_t *xq, *xs, *w;
  void* out;
  int M, N, K, Kc;
  bool out_bf16;
  int tiles_n, tiles_m;
  SplitK split;
};

constexpr int kRowsWaves = 8;

template <int kTT, int kSrc>
__global__ __launch_bounds__(64 * kRowsWaves) void mx_rows_kernel(MxGemmArgs a) {
  __shared__ f32x4_t red[mx_rows_red<kTT, kRowsWaves>];
  __shared__ __attribute__((aligned(16))) uint8_t pass[kSrc == kMxRowsQ ? 16 : kRowsWaves * kTT * kMxPass];
  __shared__ int last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int tiles = a.tiles_n * a.tiles_m, part = blockIdx.x / tiles, tile = blockIdx.x - part * tiles;
  const int rb = tile % a.tiles_n, t0 = tile / a.tiles_n * 16 * kTT;
  MxRowsTile p = {a.w + static_cast<size_t>(rb) * a.Kc * kMxTileBytes, a.Kc, 0, 0, t0, a.M};
  part_range(a.Kc, a.split.parts, part, p.c0, p.c1);
  f32x4_t sum[1];
  mx_rows_body<kTT, kRowsWaves, (kTT == 2 && kSrc == kMxRowsFp32 ? 1 : 2), kSrc>(
      p, a.x, a.K, a.xq, a.xs, [](int t) { return t; }, pass, red, sum[0]);
  if (!join_parts(a.split, tile, part, true, sum, &last)) return;
  const int token = t0 + (wave % kTT) * 16 + (lane & 15), n0 = (4 * rb + wave / kTT) * 16 + 4 * (lane >> 4);
  if (token < a.M && wave < 4 * kTT)
    store4<true>(a.out, static_cast<size_t>(token) * a.N + n0, a.N - n0, sum[0], a.out_bf16);
}

// a tile of up to 32 kT kWM rows from m0 on, on the narrowest instance that holds them
template <int kT, int kWN, int kWM, bool kSplit>
__device__ __forceinline__ void gemm_tile(const MxGemmArgs& a, int tn, int m0, int rows, int part, int tile,
                                          uint8_t* lds) {
  using S = MxTileShape<kT, kWN, kWM>;
  if constexpr (kT > 1) {
    if (rows <= 32 * (kT - 1) * kWM) {
      gemm_tile<kT - 1, kWN, kWM, kSplit>(a, tn, m0, rows, part, tile, lds);
      return;
    }
  }
  const int wave = threadIdx.x >> 6, wn = wave % kWN, wm = wave / kWN;
  MxTile p;
  p.w = a.w;
  p.rb0 = tn * (S::BN / 64);
  p.row_blocks = mx_row_blocks(a.N);
  p.xq = a.xq + static_cast<size_t>(m0) * a.Kc * 64;
  p.xs = a.xs + static_cast<size_t>(m0) * a.Kc * 4;
  p.xq_bytes = static_cast<uint32_t>(rows) * a.Kc * 64;
  p.xs_bytes = static_cast<uint32_t>(rows) * a.Kc * 4;
  p.Kc = a.Kc;
  p.c0 = 0;
  p.c1 = a.Kc;
  if constexpr (kSplit) part_range(a.Kc, a.split.parts, part, p.c0, p.c1);
  f32x16_t acc[kQ][kT];
  mx_tile_body<kT, kWN, kWM>(p, [&](int i) { return min(i, rows - 1); }, lds, acc);
  if constexpr (kSplit) {
    f32x4_t(&v)[4 * kQ * kT] = reinterpret_cast<f32x4_t(&)[4 * kQ * kT]>(acc);
    if (!join_parts(a.split, tile, part, true, v, reinterpret_cast<int*>(lds))) return;
    __syncthreads();  // everyone has read the word of LDS
  }
  const int n0 = tn * S::BN + wn * 32 * kQ, w0 = wm * 32 * kT;
  const auto row_of = [&](int row, auto type) -> decltype(type)* {
    return w0 + row < rows ? static_cast<decltype(type)*>(a.out) + static_cast<size_t>(m0 + w0 + row) * a.N + n0
                           : nullptr;
  };
  if (a.out_bf16)
    mx_store_tile<uint16_t>(lds, acc, [&](int row) { return row_of(row, uint16_t()); }, a.N - n0);
  else
    mx_store_tile<float>(lds, acc, [&](int row) { return row_of(row, float()); }, a.N - n0);
}

// tiles of 64 kWN weight rows x kBM rows, kBM + kOver = 32 kT kWM: the last one takes up
// to kOver rows more (mx_tile.h)
template <int kT, int kWN, int kWM, int kOver, bool kSplit>
__global__ __launch_bounds__(64 * kWN * kWM, 2) void mx_tile_kernel(MxGemmArgs a) {
  using S = MxTileShape<kT, kWN, kWM>;
  constexpr int kBM = S::BM - kOver;
  __shared__ __attribute__((aligned(128))) uint8_t lds[S::kLds];
  const int tiles = a.tiles_n * a.tiles_m, part = kSplit ? blockIdx.x / tiles : 0;
  int tn, tm;
  mx_tile_at(mx_xcd_tile(blockIdx.x - part * tiles, tiles), a.tiles_n, a.tiles_m, tn, tm);
  const int m0 = tm * kBM, rows = tm == a.tiles_m - 1 ? a.M - m0 : kBM;
  gemm_tile<kT, kWN, kWM, kSplit>(a, tn, m0, rows, part, tm * a.tiles_n + tn, lds);
}

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// K parts that bring the workgroups to the number of CUs, each with at least `least` chunks
int split_parts(int tiles, int Kc, int least) {
  if (tiles > kSplitTiles) return 1;
  int p = 256 / tiles;
  p = p < Kc / least ? p : Kc / least;
  return p < 1 ? 1 : p;
}

// How a product of these sizes runs: the kernel, and its K parts. Measured, us, the product
// alone; (p): K parts.
//
// Registers (mx_rows.h) up to 32 rows: N = 4096, K = 7168, registers (4) / tiles of 64 x 64 (4):
// M = 16 6.9 / 10.0, M = 32 8.4 / 10.2. They quantise the rows as well (moe_mx_proj in one
// launch), so they also take more rows while that gives at most one workgroup a CU, of at
// most 18 chunks (two or three a wave). moe_mx_proj, us, registers / quantise and tiles: M =
// 256, N = 512, K = 1024 4.5 / 8.6; M = 64, N = 4096, K = 2048 8.7 / 11.1; M = 1000, N = 64, K =
// 4096 8.0 (4) / 12.4; on two workgroups a CU M = 512, N = 2048, K = 1024 9.6 / 7.6; of 32
// chunks M = 64, N = 4096, K = 4096 14.4 / 13.3. 16 rows a workgroup while that keeps to one a
// CU, else 32: M = 64, N = 2048, K = 2048 16 rows 5.8, 32 rows 8.6. Parts cost about 2 us to add
// up: M = 1 9.8 (1), 8.6 (2), 7.8 (4); M = 1, N = 7168, K = 2048 5.3 (1), 6.7 (2); M = 8, N =
// 1024, K = 4096 7.8 (1), 6.3 (4).
//
// Tiles of 64 x 64 (four workgroups a CU) while they are at most 512, of 128 x 128 (two) or
// 256 x 256 (one, its last row tile up to 320 rows) beyond, by rounds over the CUs. 64 / 128 /
// 256: M = 128, N = 7168, K = 2048 6.2 / 7.7 / 9.9; M = 512, N = 4096, K = 7168 18.4 / 18.9 /
// 37; M = 1024 - / 26 / 39, M = 2048 - / 41 / 45, M = 4096 - / 78 / 62, M = 8192 - / 147 / 117;
// 3000 x 3000 x 3000 - / 26 / 24. K parts of 64 x 64 tiles: M = 64, N = 4096, K = 7168 13.2 (1),
// 10.9 (2), 10.2 (4); M = 128, N = 512, K = 8192 14.4 (1), 9.1 (4), 9.7 (8); M = 40, N = 256, K =
// 2048 5.8 (1), 6.6 (2).
enum Form { kRows16, kRows32, kTile64, kTile128, kTile256 };
struct Plan {
  Form form;
  int tiles_n, tiles_m, parts;
  size_t part_bytes;  // fp32 sums of one part of one tile
};

Plan mx_plan(const moe_mx_dims& m) {
  const int Kc = mx_chunks(m.K);
  Plan p;
  p.tiles_n = mx_row_blocks(m.N);
  p.form = p.tiles_n * ceil_div(m.M, 16) <= 256 || m.M <= 16 ? kRows16 : kRows32;
  p.tiles_m = ceil_div(m.M, p.form == kRows16 ? 16 : 32);
  p.parts = split_parts(p.tiles_n * p.tiles_m, Kc, Kc >= 32 ? 8 : 16);
  if (m.M <= 32 || (p.tiles_n * p.tiles_m <= 256 && ceil_div(Kc, p.parts) <= 18)) {
    p.part_bytes = 64 * kRowsWaves * 16;
    return p;
  }
  p.parts = 1;
  p.part_bytes = 0;
  const auto tiles = [&](Form form, int tn, int tm) {
    p.form = form;
    p.tiles_n = tn;
    p.tiles_m = tm;
    return static_cast<size_t>(tn) * tm;
  };
  if (tiles(kTile64, mx_row_blocks(m.N), mx_row_tiles<64, 0>(m.M)) <= 512) {
    p.parts = split_parts(p.tiles_n * p.tiles_m, Kc, 12);
    p.part_bytes = 8 * 128 * 16;
    return p;
  }
  const size_t r128 = (tiles(kTile128, ceil_div(m.N, 128), mx_row_tiles<128, 0>(m.M)) + 511) / 512;
  const Plan small = p;
  const size_t r256 = (tiles(kTile256, ceil_div(m.N, 256), mx_row_tiles<256, 64>(m.M)) + 255) / 256;
  return r128 * 66 <= r256 * 100 ? small : p;
}

size_t gemm_workspace(const moe_mx_dims& m) {
  const Plan p = mx_plan(m);
  return kSplitCounterBytes +
         (p.parts > 1 ? static_cast<size_t>(p.tiles_n) * p.tiles_m * p.parts * p.part_bytes : 0);
}

template <int kSrc>
void launch_rows(const MxGemmArgs& a, const Plan& p, unsigned grid, hipStream_t stream) {
  if (p.form == kRows16)
    mx_rows_kernel<1, kSrc><<<grid, 64 * kRowsWaves, 0, stream>>>(a);
  else
    mx_rows_kernel<2, kSrc><<<grid, 64 * kRowsWaves, 0, stream>>>(a);
}

inline bool takes_rows(const Plan& p) { return p.form == kRows16 || p.form == kRows32; }

// x: the rows themselves (where the kernel takes them), else NULL
void launch_gemm(const moe_mx_dims& m, const void* x, const uint8_t* xq, const uint8_t* xs,
                 const void* packed, void* out, void* workspace, hipStream_t stream) {
  const Plan p = mx_plan(m);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const MxGemmArgs a = {x,
                        xq,
                        xs,
                        static_cast<const uint8_t*>(packed),
                        out,
                        m.M,
                        m.N,
                        m.K,
                        mx_chunks(m.K),
                        m.out_type == MOE_BF16,
                        p.tiles_n,
                        p.tiles_m,
                        SplitK{p.parts, reinterpret_cast<int32_t*>(ws),
                               reinterpret_cast<f32x4_t*>(ws + kSplitCounterBytes)}};
  const unsigned grid = static_cast<unsigned>(p.tiles_n) * p.tiles_m * p.parts;
  if (p.form == kTile256)
    mx_tile_kernel<5, 4, 2, 64, false><<<grid, 512, 0, stream>>>(a);
  else if (p.form == kTile128)
    mx_tile_kernel<2, 2, 2, 0, false><<<grid, 256, 0, stream>>>(a);
  else if (p.form == kTile64)
    mx_tile_kernel<1, 1, 2, 0, true><<<grid, 128, 0, stream>>>(a);
  else if (!x)
    launch_rows<kMxRowsQ>(a, p, grid, stream);
  else if (m.in_type == MOE_BF16)
    launch_rows<kMxRowsBf16>(a, p, grid, stream);
  else
    launch_rows<kMxRowsFp32>(a, p, grid, stream);
}

size_t codes_bytes(const moe_mx_dims& m) {
  return round_up(static_cast<size_t>(m.M) * mx_chunks(m.K) * 64, 256);
}
size_t scales_bytes(const moe_mx_dims& m) {
  return round_up(static_cast<size_t>(m.M) * mx_chunks(m.K) * 4, 256);
}

void launch_quant(const moe_mx_dims& m, const void* x, uint8_t* q, uint8_t* s, hipStream_t stream) {
  const int Kc = mx_chunks(m.K);
  const unsigned grid = static_cast<unsigned>((static_cast<size_t>(m.M) * Kc * 8 + 255) / 256);
  if (m.in_type == MOE_BF16)
    mx_quant_kernel<uint16_t><<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x), q, s, m.M, m.K, Kc);
  else
    mx_quant_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), q, s, m.M, m.K, Kc);
}

}  // namespace

int check_mx_dims(const moe_mx_dims* d) {
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL);
  MOE_REQUIRE(d->M >= 1 && d->M <= 262144, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->N >= 1 && d->N <= 32768, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->K >= 1 && d->K <= 32768, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->in_type == MOE_BF16 || d->in_type == MOE_FP32, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(d->out_type == MOE_BF16 || d->out_type == MOE_FP32, MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

}  // namespace moeblk

using namespace moeblk;

extern "C" {

int moe_check_mx_dims(const moe_mx_dims* dims) { return check_mx_dims(dims); }

int moe_mx_quant(const moe_mx_dims* dims, const void* x, void* q, void* scales,
                 hipStream_t stream) {
  const int rc = check_mx_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(x && q && scales, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(x) && aligned16(q) && aligned16(scales), MOE_ERR_ALIGN);
  launch_quant(*dims, x, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales), stream);
  return launch_status();
}

int moe_mx_dequant(const moe_mx_dims* dims, const void* q, const void* scales, void* x,
                   hipStream_t stream) {
  const int rc = check_mx_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(q && scales && x, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(q) && aligned16(scales) && aligned16(x), MOE_ERR_ALIGN);
  const int Kc = mx_chunks(dims->K);
  const uint8_t *qb = static_cast<const uint8_t*>(q), *sb = static_cast<const uint8_t*>(scales);
  const int per_row = ceil_div(dims->K, dims->out_type == MOE_BF16 ? 8 : 4);
  const unsigned grid = static_cast<unsigned>((static_cast<size_t>(dims->M) * per_row + 255) / 256);
  if (dims->out_type == MOE_BF16)
    mx_dequant_kernel<uint16_t><<<grid, 256, 0, stream>>>(qb, sb, static_cast<uint16_t*>(x), dims->M, dims->K, Kc);
  else
    mx_dequant_kernel<float><<<grid, 256, 0, stream>>>(qb, sb, static_cast<float*>(x), dims->M, dims->K, Kc);
  return launch_status();
}

size_t moe_packed_mx_bytes(const moe_mx_dims* dims) {
  return check_mx_dims(dims) ? 0 : mx_packed_bytes(dims->N, dims->K);
}

int moe_pack_mx(const moe_mx_dims* dims, const void* q, const void* scales, void* packed,
                hipStream_t stream) {
  const int rc = check_mx_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(q && scales && packed, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(q) && aligned16(scales) && aligned16(packed), MOE_ERR_ALIGN);
  const int Kc = mx_chunks(dims->K);
  mx_pack_kernel<<<mx_row_blocks(dims->N) * Kc, 256, 0, stream>>>(
      static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(scales),
      static_cast<uint8_t*>(packed), dims->N, dims->K, Kc);
  return launch_status();
}

size_t moe_mx_gemm_workspace_bytes(const moe_mx_dims* dims) {
  return check_mx_dims(dims) ? 0 : gemm_workspace(*dims);
}

int moe_mx_gemm(const moe_mx_dims* dims, const void* xq, const void* xs, const void* w_packed,
                void* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_mx_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(xq && xs && w_packed && out && workspace, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(xq) && aligned16(xs) && aligned16(w_packed) && aligned16(out) &&
                  aligned16(workspace),
              MOE_ERR_ALIGN);
  MOE_REQUIRE(workspace_bytes >= gemm_workspace(*dims), MOE_ERR_WORKSPACE);
  launch_gemm(*dims, nullptr, static_cast<const uint8_t*>(xq), static_cast<const uint8_t*>(xs),
              w_packed, out, workspace, stream);
  return launch_status();
}

size_t moe_mx_proj_workspace_bytes(const moe_mx_dims* dims) {
  return check_mx_dims(dims) ? 0 : gemm_workspace(*dims) + codes_bytes(*dims) + scales_bytes(*dims);
}

int moe_mx_proj(const moe_mx_dims* dims, const void* x, const void* w_packed, void* out,
                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_mx_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(x && w_packed && out && workspace, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(x) && aligned16(w_packed) && aligned16(out) && aligned16(workspace),
              MOE_ERR_ALIGN);
  MOE_REQUIRE(workspace_bytes >= moe_mx_proj_workspace_bytes(dims), MOE_ERR_WORKSPACE);
  if (takes_rows(mx_plan(*dims))) {
    launch_gemm(*dims, x, nullptr, nullptr, w_packed, out, workspace, stream);
  } else {
    uint8_t* q = static_cast<uint8_t*>(workspace) + gemm_workspace(*dims);
    uint8_t* s = q + codes_bytes(*dims);
    launch_quant(*dims, x, q, s, stream);
    launch_gemm(*dims, nullptr, q, s, w_packed, out, workspace, stream);
  }
  return launch_status();
}

}  // extern "C"
