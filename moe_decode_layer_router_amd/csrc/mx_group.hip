// mx_group.hip -- the experts' MXFP4 products of many rows: gate_up with SwiGLU from
// the tokens' quantised rows (moe_mx_gate_up), and down (moe_mx_down).
//
// The rows are sorted by expert (moe_sort): expert e has rows offsets[e] ..
// offsets[e + 1] - 1, as the device knows; the host sizes the grid for any split of
// the picks, and a workgroup finds its tile from the offsets or ends. The weights are
// those that moe_pack_mxfp4 lays out for the decode path.
//
// In gate_up a lane's four outputs of a row tile are (gate i, gate i + 1, up i,
// up i + 1) (common.h), so SwiGLU needs no exchange; a row block of 64 weight rows is
// 32 intermediates, one MX block of the result, whose 32 values lie in four lanes: the
// next product's quantisation is two exchanges away.
#include <type_traits>

#include "host.h"
#include "mx_dev.h"
#include "mx_rows.h"
#include "mx_tile.h"

namespace moeblk {
namespace {

constexpr int kMaxGroups = 32;

struct MxGroupArgs {
  const uint8_t *xq, *xs, *w;
  const int32_t *offsets, *rows;  // rows: gate_up's row -> token, NULL: the rows themselves
  void* out;
  uint8_t* hs;  // scale bytes of an MXFP4 result
  int T, R, n, N, Kc;
  int type;  // MOE_BF16, MOE_FP32 or MOE_MXFP4
  size_t w_bytes;  // an expert's
};

struct Group {
  int e, first, count, tile;  // expert, its first row and rows; the tile within it (-1: none)
};

// Tile `t` of all experts' (tiles_n a group of kBM rows). Lane i holds expert i; offsets
// outside the rows are taken as the nearer end.
template <int kBM, int kOver>
__device__ __forceinline__ Group find_group(const MxGroupArgs& a, int b, int tiles_n) {
  const int lane = threadIdx.x & 63;
  const int o = lane <= a.n ? min(max(a.offsets[lane], 0), a.R) : 0;
  const int next = __shfl_down(o, 1, kWave);
  const int count = lane < a.n ? max(next - o, 0) : 0;
  const int tiles = mx_row_tiles<kBM, kOver>(count) * tiles_n;
  int incl = tiles;
#pragma unroll
  for (int s = 1; s < kMaxGroups; s <<= 1) {
    const int v = __shfl_up(incl, s, kWave);
    if (lane >= s) incl += v;
  }
  const int total = __builtin_amdgcn_readlane(incl, kMaxGroups - 1);
  Group g;
  const int t = mx_xcd_tile(b, total);
  if (t < 0) {
    g.e = g.first = g.count = 0;
    g.tile = -1;
    return g;
  }
  const uint64_t m = __ballot(t < incl && lane < kMaxGroups);
  g.e = __builtin_ctzll(m);
  g.first = __builtin_amdgcn_readlane(o, g.e);
  g.count = __builtin_amdgcn_readlane(count, g.e);
  g.tile = t - __builtin_amdgcn_readlane(incl - tiles, g.e);
  return g;
}

// ---------------------------------------------------------------- many rows an expert

// a tile of an expert's rows: `rows` of them from `first` on, up to 32 kT kWM
template <int kT, int kWN, int kWM, bool kGateUp>
__device__ __forceinline__ void group_tile(const MxGroupArgs& a, const Group& gr, int tn, int first,
                                           int rows, uint8_t* lds) {
  using S = MxTileShape<kT, kWN, kWM>;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m32 = lane & 31, hi = lane >> 5;
  const int wn = wave % kWN, wm = wave / kWN;
  MxTile p;
  p.w = a.w + gr.e * a.w_bytes;
  p.rb0 = tn * (S::BN / 64);
  p.row_blocks = a.N / kRowsPerBlock;
  const size_t base = kGateUp ? 0 : first;
  const uint32_t readable = kGateUp ? a.T : rows;
  p.xq = a.xq + base * a.Kc * 64;
  p.xs = a.xs + base * a.Kc * 4;
  p.xq_bytes = readable * a.Kc * 64u;
  p.xs_bytes = readable * a.Kc * 4u;
  p.Kc = a.Kc;
  p.c0 = 0;
  p.c1 = a.Kc;
  f32x16_t acc[kQ][kT];
  mx_tile_body<kT, kWN, kWM>(
      p,
      [&](int i) {
        i = min(i, rows - 1);
        if constexpr (kGateUp) return min(max(a.rows[first + i], 0), a.T - 1);
        return i;
      },
      lds, acc);
  const int m0 = wm * 32 * kT;  // of this wave
  const auto row_of = [&](int row, auto type, int width, int col) -> decltype(type)* {
    return m0 + row < rows
               ? static_cast<decltype(type)*>(a.out) + static_cast<size_t>(first + m0 + row) * width + col
               : nullptr;
  };
  if constexpr (kGateUp) {
    // elements 4 j .. 4 j + 3 are (gate i, gate i + 1, up i, up i + 1) of i = 16 q + 4 j + 2 hi
    const int I = a.N / 2, i0 = (p.rb0 + wn) * 32;  // first intermediate of this wave
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[q][t][4 * j] = mx_swiglu(acc[q][t][4 * j], acc[q][t][4 * j + 2]);
          acc[q][t][4 * j + 1] = mx_swiglu(acc[q][t][4 * j + 1], acc[q][t][4 * j + 3]);
        }
    if (a.type == MOE_BF16) {
      mx_store<uint16_t, kT, 16 * kQ>(
          lds,
          [&](int t, uint8_t* o) {
#pragma unroll
            for (int q = 0; q < kQ; ++q)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t*>(o + q * 32 + j * 8 + 4 * hi) =
                    mx_bf16x2(acc[q][t][4 * j], acc[q][t][4 * j + 1]);
          },
          [&](int row) { return row_of(row, uint16_t(), I, i0); }, I - i0);
      return;
    }
    // MXFP4: a block is the two 32-row units, 16 values of a lane and 16 of lane ^ 32; its codes
    // meet in LDS, 16 bytes a row (8192 tokens, 32 experts of 4096 x 2048: 108 us, the bf16 result
    // 110)
    uint8_t* o = lds + wave * (32 * kT * 16);
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const int row = m0 + t * 32 + m32;
      float v[2][8];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i >> 3][i & 7] = acc[i >> 3][t][4 * ((i & 7) >> 1) + (i & 1)];
        m = max(m, __float_as_uint(v[i >> 3][i & 7]) & 0x7fffffffu);
      }
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32, kWave)));
      const uint32_t byte = mx_scale_byte(m);
      const float s = e8m0_scale(byte);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = mx_codes_or_zero(mx_codes(v[h], s), byte);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[(t * 32 + m32) * 16 + 8 * h + 2 * j + hi] = static_cast<uint8_t>(c >> (8 * j));
      }
      if (hi == 0 && row < rows && i0 < I)
        a.hs[static_cast<size_t>(first + row) * (I / 32) + i0 / 32] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (32 * kT + 63) / 64; ++i) {
      const int at = i * 64 + lane, row = m0 + at;
      if (at < 32 * kT && row < rows && i0 < I)
        *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(a.out) +
                                    static_cast<size_t>(first + row) * (I / 2) + i0 / 2) =
            *reinterpret_cast<const u32x4_t*>(o + at * 16);
    }
  } else {
    const int n0 = tn * S::BN + wn * 32 * kQ;
    if (a.type == MOE_BF16)
      mx_store_tile<uint16_t>(lds, acc, [&](int row) { return row_of(row, uint16_t(), a.N, n0); }, a.N - n0);
    else
      mx_store_tile<float>(lds, acc, [&](int row) { return row_of(row, float(), a.N, n0); }, a.N - n0);
  }
}

// A tile of `rows` rows runs on the narrowest instance that holds them, in steps of 32 kWM:
// fewer MFMAs, down to where the weights' copies are its time.
template <int kT, int kWN, int kWM, bool kGateUp>
__device__ __forceinline__ void group_tile_rows(const MxGroupArgs& a, const Group& gr, int tn, int first,
                                                int rows, uint8_t* lds) {
  if constexpr (kT > 1) {
    if (rows <= 32 * (kT - 1) * kWM) {
      group_tile_rows<kT - 1, kWN, kWM, kGateUp>(a, gr, tn, first, rows, lds);
      return;
    }
  }
  group_tile<kT, kWN, kWM, kGateUp>(a, gr, tn, first, rows, lds);
}

// tiles of 64 kWN weight rows x kBM rows, kBM + kOver = 32 kT kWM
template <int kT, int kWN, int kWM, int kOver, bool kGateUp>
__global__ __launch_bounds__(64 * kWN * kWM, 2) void mx_group_tile_kernel(MxGroupArgs a) {
  using S = MxTileShape<kT, kWN, kWM>;
  constexpr int kBM = S::BM - kOver;
  __shared__ __attribute__((aligned(128))) uint8_t lds[S::kLds];
  const int tiles_n = (a.N + S::BN - 1) / S::BN;
  const Group gr = find_group<kBM, kOver>(a, blockIdx.x, tiles_n);
  if (gr.tile < 0) return;
  const int tiles_m = mx_row_tiles<kBM, kOver>(gr.count);
  int tn, tm;
  mx_tile_at(gr.tile, tiles_n, tiles_m, tn, tm);
  const int rows = tm == tiles_m - 1 ? gr.count - tm * kBM : kBM;
  group_tile_rows<kT, kWN, kWM, kGateUp>(a, gr, tn, gr.first + tm * kBM, rows, lds);
}

// ---------------------------------------------------------------- few rows of few experts
//
// A workgroup takes one row block and 16 rows of an expert, weights straight into registers
// (mx_rows.h).
constexpr int kFewRows = 16, kFewWaves = 8;

template <bool kGateUp>
__global__ __launch_bounds__(64 * kFewWaves) void mx_group_few_kernel(MxGroupArgs a) {
  __shared__ f32x4_t red[mx_rows_red<1, kFewWaves>];
  const int blocks = a.N / kRowsPerBlock;
  const Group gr = find_group<kFewRows, 0>(a, blockIdx.x, blocks);
  if (gr.tile < 0) return;
  const int tiles_m = mx_row_tiles<kFewRows, 0>(gr.count);
  const int rb = gr.tile / tiles_m, m0 = gr.tile % tiles_m * kFewRows;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const MxRowsTile p = {a.w + gr.e * a.w_bytes + static_cast<size_t>(rb) * a.Kc * kMxTileBytes, a.Kc, 0, a.Kc,
                        m0, gr.count};
  f32x4_t sum;  // waves 0 .. 3: of row tile `wave`
  mx_rows_body<1, kFewWaves, 2, kMxRowsQ>(
      p, nullptr, 0, a.xq, a.xs,
      [&](int i) {
        if constexpr (kGateUp) return min(max(a.rows[gr.first + i], 0), a.T - 1);
        return gr.first + i;
      },
      nullptr, red, sum);
  if constexpr (!kGateUp) {
    const int row = m0 + m16, n = (4 * rb + wave) * 16 + 4 * g;
    if (wave < 4 && row < gr.count)
      store4<true>(a.out, static_cast<size_t>(gr.first + row) * a.N + n, a.N - n, sum, a.type == MOE_BF16);
  } else {
    // the 32 intermediates of a row meet in LDS; then 4 threads a row, 8 values each
    constexpr int kPitch = 36;
    float* h = reinterpret_cast<float*>(red);
    __syncthreads();  // the sums have been read
    if (wave < 4) {
      float* to = h + m16 * kPitch + 8 * wave + 2 * g;
      to[0] = mx_swiglu(sum[0], sum[2]);
      to[1] = mx_swiglu(sum[1], sum[3]);
    }
    __syncthreads();
    const int row = threadIdx.x >> 2, j = threadIdx.x & 3, I = a.N / 2;
    if (row >= kFewRows || m0 + row >= gr.count) return;  // all four threads of a row
    const float* from = h + row * kPitch + 8 * j;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = from[i];
    const size_t at = static_cast<size_t>(gr.first + m0 + row);
    if (a.type == MOE_BF16) {
      u32x4_t q;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = mx_bf16x2(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + at * I + 32 * rb + 8 * j) = q;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1, kWave)));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2, kWave)));
      const uint32_t byte = mx_scale_byte(m);
      const uint32_t q = mx_codes_or_zero(mx_codes(v, e8m0_scale(byte)), byte);
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + at * (I / 2) + 16 * rb + 4 * j) = q;
      if (j == 0) a.hs[at * (I / 32) + rb] = static_cast<uint8_t>(byte);
    }
  }
}

// ---------------------------------------------------------------- host

// most tiles of kBM rows that R rows of n experts can make
inline int64_t max_tiles(int64_t R, int n, int bm) {
  const int64_t groups = n < R ? n : R;
  return (R - groups) / bm + groups;
}

// One kernel serves every expert of a call; which one follows from what the host knows, the
// rows an expert has on average (evenly popular experts) and the experts that have any.
// Measured, us, gate_up of 4096 x 2 x 2048, 32 of 256 experts held, top-8, tiles of 128 x 128 /
// 256 x 256: 2 rows an expert 41.5 / 42.6, 16 rows 50.5 / 48.1, 32 rows 55 / 50, 64 rows 73 / 56,
// 256 rows 138 / 105; seven experts of one row 14.2 / 16.4.
// Few experts, or narrow ones, leave most CUs without a large tile: there tiles of 64 x 64,
// and for up to 16 rows the register kernel, which splits K over its waves. One expert,
// 128 x 128 / 64 x 64 / registers: 1 row 10.3 / 9.5 / 4.9, 16 rows 10.4 / 9.6 / 6.1, 64 rows 10.6 /
// 9.7 / -, 100 rows 12.9 / 9.7 / -.
//
// The grid is sized for any split of the picks, all of them local included, so that with 32 of 256
// experts held seven of eight workgroups of 8192 tokens find no tile, behind those that do. The
// same rows where the grid fits them (1024 tokens, 32 of 32 held), us: gate_up with a bf16 result 110 ->
// 109, with an MXFP4 one 108 -> 97, down 65 -> 59.
enum GroupForm { kGroupFew, kGroup64, kGroup128, kGroup256 };

GroupForm group_form(const moe_mx_group_dims& m, int N) {
  const int64_t picks = static_cast<int64_t>(m.T) * m.topk * m.n_local / m.E;  // that are local
  const int64_t per = static_cast<int64_t>(m.T) * m.topk / m.E;
  const int64_t active = picks < 1 ? 1 : picks < m.n_local ? picks : m.n_local;
  const int64_t blocks = active * (N / kRowsPerBlock), tiles64 = blocks * ((per + 63) / 64);
  const int64_t tiles256 = active * ((N + 255) / 256) * (per < 384 ? 1 : (per + 128) / 256);
  if (blocks <= 256 && per <= kFewRows) return kGroupFew;
  if (per >= 12 && tiles256 >= 200) return kGroup256;
  return tiles64 <= 512 ? kGroup64 : kGroup128;
}

template <bool kGateUp>
void launch_group(const moe_mx_group_dims& m, const MxGroupArgs& a, hipStream_t stream) {
  const auto grid = [&](int bm, int bn) {
    return static_cast<unsigned>(max_tiles(a.R, a.n, bm) * ((a.N + bn - 1) / bn));
  };
  switch (group_form(m, a.N)) {
    case kGroupFew:
      mx_group_few_kernel<kGateUp><<<grid(kFewRows, 64), 64 * kFewWaves, 0, stream>>>(a);
      break;
    case kGroup64:
      mx_group_tile_kernel<1, 1, 2, 0, kGateUp><<<grid(64, 64), 128, 0, stream>>>(a);
      break;
    case kGroup128:
      mx_group_tile_kernel<2, 2, 2, 0, kGateUp><<<grid(128, 128), 256, 0, stream>>>(a);
      break;
    case kGroup256:
      mx_group_tile_kernel<5, 4, 2, 64, kGateUp><<<grid(256, 256), 512, 0, stream>>>(a);
      break;
  }
}

}  // namespace

int check_mx_group_dims(const moe_mx_group_dims* d) {
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL);
  MOE_REQUIRE(d->T >= 1 && d->T <= 262144, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->E >= 1 && d->E <= 256, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->topk >= 1 && d->topk <= 8 && d->topk <= d->E, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->n_local >= 1 && d->n_local <= kMaxGroups && d->n_local <= d->E, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->d >= 128 && d->d <= 16384 && d->d % 128 == 0, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->I >= 128 && d->I <= 8192 && d->I % 128 == 0, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->h_type == MOE_BF16 || d->h_type == MOE_MXFP4, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(d->out_type == MOE_BF16 || d->out_type == MOE_FP32, MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

}  // namespace moeblk

using namespace moeblk;

extern "C" {

int moe_check_mx_group_dims(const moe_mx_group_dims* dims) { return check_mx_group_dims(dims); }

// The kernel that a product with N weight rows an expert takes (GroupForm), for tests: no part
// of the interface.
int moeblk_mx_group_form(const moe_mx_group_dims* dims, int N) {
  return check_mx_group_dims(dims) ? -1 : group_form(*dims, N);
}

int moe_mx_gate_up(const moe_mx_group_dims* dims, const void* xq, const void* xs,
                   const int32_t* offsets, const int32_t* rows, const void* w13_packed, void* h,
                   void* hs, hipStream_t stream) {
  const int rc = check_mx_group_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(xq && xs && offsets && rows && w13_packed && h, MOE_ERR_NULL);
  MOE_REQUIRE(hs || dims->h_type != MOE_MXFP4, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(xq) && aligned16(xs) && aligned16(offsets) && aligned16(rows) &&
                  aligned16(w13_packed) && aligned16(h) && aligned16(hs),
              MOE_ERR_ALIGN);
  const int N = 2 * dims->I;
  const MxGroupArgs a = {static_cast<const uint8_t*>(xq),
                         static_cast<const uint8_t*>(xs),
                         static_cast<const uint8_t*>(w13_packed),
                         offsets,
                         rows,
                         h,
                         static_cast<uint8_t*>(hs),
                         dims->T,
                         dims->T * dims->topk,
                         dims->n_local,
                         N,
                         mx_chunks(dims->d),
                         dims->h_type,
                         mx_packed_bytes(N, dims->d)};
  launch_group<true>(*dims, a, stream);
  return launch_status();
}

int moe_mx_down(const moe_mx_group_dims* dims, const void* hq, const void* hs,
                const int32_t* offsets, const void* w2_packed, void* y, hipStream_t stream) {
  const int rc = check_mx_group_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(hq && hs && offsets && w2_packed && y, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(hq) && aligned16(hs) && aligned16(offsets) && aligned16(w2_packed) &&
                  aligned16(y),
              MOE_ERR_ALIGN);
  const MxGroupArgs a = {static_cast<const uint8_t*>(hq),
                         static_cast<const uint8_t*>(hs),
                         static_cast<const uint8_t*>(w2_packed),
                         offsets,
                         nullptr,
                         y,
                         nullptr,
                         dims->T,
                         dims->T * dims->topk,
                         dims->n_local,
                         dims->d,
                         mx_chunks(dims->I),
                         dims->out_type,
                         mx_packed_bytes(dims->d, dims->I)};
  launch_group<false>(*dims, a, stream);
  return launch_status();
}

}  // extern "C"
