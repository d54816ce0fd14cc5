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
// one DPP step for the maximum, 8 bytes of codes a lane.

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

// 8 columns a thread: 4 bytes of codes
template <typename T>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ s,
                                                         T* __restrict__ x, int M, int K, int Kc) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
  const size_t item = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  const int per_row = (K + 7) / 8;
  const size_t row = item / per_row;
  const int c = static_cast<int>(item - row * per_row) * 8;
  if (row >= static_cast<size_t>(M)) return;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(q + row * (static_cast<size_t>(Kc) * 64) + c / 2);
  const float sc = e8m0_scale(s[row * (static_cast<size_t>(Kc) * 4) + c / kMxBlock]);
  T* o = x + row * K + c;
  if constexpr (sizeof(T) == 4) {
    const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 0);
    const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 1);
    const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 2);
    const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 3);
    const float v[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    if (c + 8 <= K) {
      *reinterpret_cast<f32x4_any_t*>(o) = f32x4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_any_t*>(o + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (c + i < K) o[i] = v[i];
    }
  } else {
    const u32x4_t v = __builtin_bit_cast(u32x4_t, decode_fp4x8(w, sc));
    if (c + 8 <= K) {
      *reinterpret_cast<u32x4_any_t*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (c + i < K) o[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
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

template <int kRT, int kTT, int kNW, int kRing, int kSrc>
__global__ __launch_bounds__(64 * kNW) void mx_rows_kernel(MxGemmArgs a) {
  constexpr int kEach = (kRT * kTT + kNW - 1) / kNW;
  __shared__ f32x4_t red[mx_rows_red<kRT, kTT, kNW>()];
  __shared__ int last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int tiles = a.tiles_n * a.tiles_m, part = blockIdx.x / tiles, tile = blockIdx.x - part * tiles;
  const int rt0 = tile % a.tiles_n * kRT, t0 = tile / a.tiles_n * 16 * kTT;
  MxRowsTile p = {a.w, rt0, a.Kc, 0, 0, t0, a.M};
  part_range(a.Kc, a.split.parts, part, p.c0, p.c1);
  f32x4_t sum[kEach];
  mx_rows_body<kRT, kTT, kNW, kRing, kSrc>(p, a.x, a.K, a.xq, a.xs, [](int t) { return t; }, red, sum);
  if (!join_parts(a.split, tile, part, true, sum, &last)) return;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kNW + wave, token = t0 + (i % kTT) * 16 + (lane & 15);
    const int n0 = (rt0 + i / kTT) * 16 + 4 * (lane >> 4);
    if (token < a.M && i < kRT * kTT)
      store4<true>(a.out, static_cast<size_t>(token) * a.N + n0, a.N - n0, sum[e], a.out_bf16);
  }
}

template <int kQ, int kT, int kWN, int kWM>
__global__ __launch_bounds__(64 * kWN * kWM, kQ * kT * kWN * kWM > 16 ? 1 : 2) void mx_tile_kernel(MxGemmArgs a) {
  using S = MxTileShape<kQ, kT, kWN, kWM>;
  __shared__ __attribute__((aligned(128))) uint8_t lds[S::kLds];
  const int wave = threadIdx.x >> 6, wn = wave % kWN, wm = wave / kWN;
  const int tiles = a.tiles_n * a.tiles_m, part = blockIdx.x / tiles;
  int tn, tm;
  mx_tile_at(mx_xcd_tile(blockIdx.x - part * tiles, tiles), a.tiles_n, a.tiles_m, tn, tm);
  const int rows = min(S::BM, a.M - tm * S::BM);
  MxTile p;
  p.w = a.w;
  p.rb0 = tn * (S::BN / 64);
  p.row_blocks = mx_row_blocks(a.N);
  p.xq = a.xq + static_cast<size_t>(tm) * S::BM * a.Kc * 64;
  p.xs = a.xs + static_cast<size_t>(tm) * S::BM * a.Kc * 4;
  p.xq_bytes = static_cast<uint32_t>(rows) * a.Kc * 64;
  p.xs_bytes = static_cast<uint32_t>(rows) * a.Kc * 4;
  p.Kc = a.Kc;
  part_range(a.Kc, a.split.parts, part, p.c0, p.c1);
  f32x16_t acc[kQ][kT];
  mx_tile_body<kQ, kT, kWN, kWM>(p, [&](int i) { return min(i, rows - 1); }, lds, acc);
  if constexpr (kQ * kT <= 4) {  // the larger tiles are never split
    f32x4_t(&v)[4 * kQ * kT] = reinterpret_cast<f32x4_t(&)[4 * kQ * kT]>(acc);
    if (!join_parts(a.split, tm * a.tiles_n + tn, part, true, v, reinterpret_cast<int*>(lds))) return;
    __syncthreads();  // everyone has read the word of LDS
  }
  const int n0 = tn * S::BN + wn * 32 * kQ, m0 = tm * S::BM + wm * 32 * kT;
  const auto row_of = [&](int row, auto type) -> decltype(type)* {
    return m0 + row < a.M ? static_cast<decltype(type)*>(a.out) + static_cast<size_t>(m0 + row) * a.N + n0
                          : nullptr;
  };
  if (a.out_bf16)
    mx_store_tile_bf16<kQ, kT>(lds, acc, [&](int row) { return row_of(row, uint16_t()); }, a.N - n0);
  else
    mx_store_tile_f32<kQ, kT>(acc, [&](int row) { return row_of(row, float()); }, a.N - n0);
}

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

int split_parts(int tiles, int Kc, int least) {
  if (tiles > kSplitTiles) return 1;
  int p = 256 / tiles;
  p = p < Kc / least ? p : Kc / least;
  return p < 1 ? 1 : p;
}

// How a product of these sizes runs: the kernel (rows: row tiles and token tiles a
// workgroup), and its K parts.
enum Form { kRows1, kRows2, kRows4, kTile128, kTile256 };
struct Plan {
  Form form;
  int rt;     // row tiles a workgroup (kRows*)
  int tiles_n, tiles_m, parts;
  size_t part_bytes;  // fp32 sums of one part of one tile
};

Plan mx_plan(const moe_mx_dims& m) {
  const int Kc = mx_chunks(m.K);
  Plan p;
  if (m.M <= 64 || ceil_div(m.N, 64) * ceil_div(m.M, 64) <= 256) {
    const int tt = m.M <= 16 ? 1 : m.M <= 32 ? 2 : 4;
    p.form = tt == 1 ? kRows1 : tt == 2 ? kRows2 : kRows4;
    p.tiles_m = ceil_div(m.M, 16 * tt);
    p.rt = tt == 1 ? (m.N <= 8192 ? 1 : 4) : ceil_div(m.N, 32) * p.tiles_m <= 256 ? 2 : 4;
    p.tiles_n = ceil_div(m.N, 16 * p.rt);
    p.parts = split_parts(p.tiles_n * p.tiles_m, Kc, tt == 1 ? 16 : 8);
    p.part_bytes = 2 * 512 * 16;
    return p;
  }
  const size_t t256 = static_cast<size_t>(ceil_div(m.N, 256)) * ceil_div(m.M, 256);
  if (t256 >= 256) {
    p.form = kTile256;
    p.tiles_n = ceil_div(m.N, 256);
    p.tiles_m = ceil_div(m.M, 256);
    p.parts = 1;
  } else {
    p.form = kTile128;
    p.tiles_n = ceil_div(m.N, 128);
    p.tiles_m = ceil_div(m.M, 128);
    p.parts = split_parts(p.tiles_n * p.tiles_m, Kc, 8);
  }
  p.part_bytes = 16 * 256 * 16;
  return p;
}

size_t gemm_workspace(const moe_mx_dims& m) {
  const Plan p = mx_plan(m);
  return kSplitCounterBytes +
         (p.parts > 1 ? static_cast<size_t>(p.tiles_n) * p.tiles_m * p.parts * p.part_bytes : 0);
}

template <int kSrc>
void launch_few(const MxGemmArgs& a, const Plan& p, unsigned grid, hipStream_t stream) {
  const auto launch = [&](auto kernel) { kernel<<<grid, 512, 0, stream>>>(a); };
  if (p.form == kRows1) {
    p.rt == 1 ? launch(mx_rows_kernel<1, 1, 8, 4, kSrc>) : launch(mx_rows_kernel<4, 1, 8, 2, kSrc>);
  } else if constexpr (kSrc == kMxRowsQ) {
    if (p.form == kRows2)
      p.rt == 2 ? launch(mx_rows_kernel<2, 2, 8, 4, kSrc>) : launch(mx_rows_kernel<4, 2, 8, 2, kSrc>);
    else
      p.rt == 2 ? launch(mx_rows_kernel<2, 4, 8, 3, kSrc>) : launch(mx_rows_kernel<4, 4, 8, 2, kSrc>);
  }
}

// x: the rows themselves (at most 16), else NULL
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
    mx_tile_kernel<4, 4, 2, 2><<<grid, 256, 0, stream>>>(a);
  else if (p.form == kTile128)
    mx_tile_kernel<2, 2, 2, 2><<<grid, 256, 0, stream>>>(a);
  else if (!x)
    launch_few<kMxRowsQ>(a, p, grid, stream);
  else if (m.in_type == MOE_BF16)
    launch_few<kMxRowsBf16>(a, p, grid, stream);
  else
    launch_few<kMxRowsFp32>(a, p, grid, stream);
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
  const unsigned grid =
      static_cast<unsigned>((static_cast<size_t>(dims->M) * ceil_div(dims->K, 8) + 255) / 256);
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
  if (mx_plan(*dims).form == kRows1) {
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
