// fp8_ffn.hip -- the expert FFNs on FP8 weights with block-128 scales
// (moe_fp8_expert_ffn), and their weight packing.
//
// gate_up + SwiGLU of every (expert, block of 64 packed rows = 32 intermediates),
// h in fp32, then down of every (expert, 64 output rows). The weights' bytes bound
// both. A workgroup's 4 waves take every fourth K block, a ring of blocks' loads in
// flight each, straight from the packed order into registers (exact form, fp8_dev.h);
// the waves' sums are added through LDS in wave order.
//
// The rows of either launch are quantised by its own workgroups, into LDS, while
// their first weight loads are in flight, in steps of up to 16 rows whose (row, K
// block) pairs fit (kFusedItems; an expert rarely has more than a few of the rows);
// else by a launch of their own in front of it.
//
// Measured (gate_up + down, us): S = 8, 7.7 active experts of 4096 x 2048 23.5 + 14.9
// (5.5, 4.3 TB/s); S = 128, 32 experts of 7168 x 2048 and a shared one 162 + 80 (5.9,
// 6.0 TB/s). With few active experts most CUs idle (K is not split): one of 4096 x 2048,
// 64 working workgroups a launch, 22 us in all for 25 MB. 4 waves instead of 8 let two or
// three workgroups share a CU, one's first loads under another's last sums: S = 8 47 -> 40
// us.
#include <type_traits>

#include "fp8_dev.h"
#include "fp8_launch.h"
#include "fp8_quant.h"
#include "host.h"

namespace moeblk {
namespace {

constexpr int kWaves = 4;  // also the row tiles of a workgroup: each wave adds up one
constexpr int kFusedRows = 16;    // most rows of a step whose workgroups quantise
constexpr int kFusedItems = 576;  // most (row, K block) pairs: two workgroups a CU
constexpr int kFewItems = 256;    // three

// rows of a launch: quantised (xq, xs), or (fused) as they are
struct RowSet {
  const void* x;      // bf16 (gate_up) or fp32 (down) rows, K columns
  const uint8_t* xq;  // e4m3 rows
  const float* xs;    // scales [Kb][rows]
  int rows;           // rows of the set
};

struct FfnArgs {
  int S, d, n_local, r_max, I, Is;
  const int32_t *counts, *offsets, *rows, *active;
  const uint8_t *w13, *w2, *ws13, *ws2;  // packed; ws*: shared expert or NULL
  RowSet x, h, hsh;                      // input rows; SwiGLU rows: routed, shared
  float *hf, *hshf;                      // fp32 SwiGLU rows: routed [r_max][I], shared [S][Is]
  uint16_t* y;
};

// LDS of a workgroup: the quantised rows, then (one token group) the waves' sums
struct Sums {
  f32x4_t v[kWaves][4][64];
};
template <int kItems>
struct FusedRows {
  uint8_t x[kItems * kFp8Block];
  float s[kItems];
};

// silu(g) u; through exp(-|g|), which does not overflow where silu(g) is still a normal number
__device__ __forceinline__ float swiglu(float g, float u) {
  const float e = expf(-fabsf(g));
  return (g < 0.0f ? g * e : g) / (1.0f + e) * u;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes),
                                           0x00020000);
}

// One block of 64 packed weight rows of an expert, all of its tokens in groups of
// 16 kTT. Lane rows 0, 1 of a D tile are gate rows and 2, 3 up rows (one scale
// each; in down the same one).
template <int kTT, bool kDown, int kItems>
__device__ __forceinline__ void ffn_block(const FfnArgs& a, bool shared, int el, int rb, int n,
                                          Sums& sums, FusedRows<kItems>& fl) {
  constexpr bool kFused = kItems > 0;
  constexpr int kRing = kTT == 1 ? 2 : 1;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  const int m16 = lane & 15, g = lane >> 4;
  const int I = shared ? a.Is : a.I;
  const int N = kDown ? a.d : 2 * I, K = kDown ? I : a.d, Kb = K / kFp8Block;
  const uint8_t* wm = kDown ? (shared ? a.ws2 : a.w2) : (shared ? a.ws13 : a.w13);
  wm += el * fp8_packed_bytes(N, K);
  const float* sc = reinterpret_cast<const float*>(wm + fp8_tile_bytes(N, K));
  const float* sw0 = sc + static_cast<size_t>(kDown ? rb / 2 : rb / 4) * Kb;
  const float* sw1 = kDown ? sw0 : sc + static_cast<size_t>(I / 128 + rb / 4) * Kb;
  const int base = shared ? 0 : a.offsets[el];
  const RowSet& set = kDown ? (shared ? a.hsh : a.h) : a.x;
  const __amdgpu_buffer_rsrc_t wr =
      rsrc(wm + static_cast<size_t>(rb) * 4 * Kb * kFp8TileBytes, 4 * Kb * kFp8TileBytes);
  const __amdgpu_buffer_rsrc_t xr = rsrc(set.xq, static_cast<size_t>(set.rows) * K);
  const __amdgpu_buffer_rsrc_t sr = rsrc(set.xs, static_cast<size_t>(set.rows) * Kb * 4);
  // row r of this expert in the row set
  const auto row_of = [&](int r) {
    return (kDown || shared) ? base + r : min(max(a.rows[base + r], 0), a.S - 1);
  };

  for (int t0 = 0; t0 < n; t0 += 16 * kTT) {
    u32x4_t w[kRing][4][2], x[kFused ? 1 : kRing][kTT][2];
    float s[kFused ? 1 : kRing][kTT], w0[kRing], w1[kRing];
    uint32_t tok[kTT];
    const auto load_w = [&](int i, int kb) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t at = static_cast<uint32_t>(r * Kb + kb) * kFp8TileBytes;
        w[i][r][0] = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16, at, kCpolNt));
        w[i][r][1] = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16, at + 1024, kCpolNt));
      }
      w0[i] = sw0[kb];
      w1[i] = sw1[kb];
    };
    const auto load_x = [&](int i, int kb) {
      if constexpr (!kFused) {
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
          const uint32_t v = tok[t] * static_cast<uint32_t>(K) + 32 * g;
          x[i][t][0] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xr, v, kb * kFp8Block, 0));
          x[i][t][1] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xr, v + 16, kb * kFp8Block, 0));
          s[i][t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                  sr, tok[t] * 4, kb * set.rows * 4, 0));
        }
      }
    };
    // the first weights are on their way before the rows are known
#pragma unroll
    for (int i = 0; i < kRing; ++i)
      if (uwave + i * kWaves < Kb) load_w(i, uwave + i * kWaves);
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const int r = min(t0 + 16 * t + m16, n - 1);
      tok[t] = kFused ? r : row_of(r);
    }
    if constexpr (kFused) {
      {  // item kb * n + r; 16-byte chunks permuted by chunk ^ (r % 8)
        using T = typename std::conditional<kDown, float, uint16_t>::type;
        const int l8 = threadIdx.x & 7;
        for (int item = threadIdx.x >> 3; item < n * Kb; item += kWaves * 8) {
          const int r = item % n, kb = item / n;
          Raw16<T> v;
          load16<T>(static_cast<const T*>(set.x) + static_cast<size_t>(row_of(r)) * K,
                          kb * kFp8Block + l8 * 16, K, v);
          float scale;
          const u32x4_t q = quant16(v, scale);
          *reinterpret_cast<u32x4_t*>(fl.x + item * kFp8Block + ((l8 ^ (r & 7)) * 16)) = q;
          if (l8 == 0) fl.s[item] = scale;
        }
        __syncthreads();
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRing; ++i)
        if (uwave + i * kWaves < Kb) load_x(i, uwave + i * kWaves);
    }

    f32x4_t acc[4][kTT];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < kTT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
    for (int first = uwave; first < Kb; first += kWaves * kRing) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) {
        const int kb = first + i * kWaves;
        if (kb < Kb) {
          constexpr bool kHold = kTT == 1;  // else the converted rows do not fit
          i32x8_t x8[kHold ? 1 : kTT];
          Bf16Frag xe[kHold ? kTT : 1];
          float s0[kTT], s1[kTT];
#pragma unroll
          for (int t = 0; t < kTT; ++t) {
            i32x8_t v;
            float f;
            if constexpr (kFused) {
              const int item = kb * n + tok[t];
              const uint8_t* p = fl.x + item * kFp8Block;
              const int sw = tok[t] & 7;
              v = join8(*reinterpret_cast<const u32x4_t*>(p + (((2 * g) ^ sw) * 16)),
                        *reinterpret_cast<const u32x4_t*>(p + (((2 * g + 1) ^ sw) * 16)));
              f = fl.s[item];
            } else {
              v = join8(x[i][t][0], x[i][t][1]);
              f = s[i][t];
            }
            s0[t] = f * w0[i];
            s1[t] = f * w1[i];
            if constexpr (kHold)
              xe[t] = e4m3_to_bf16(v);
            else
              x8[t] = v;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // one row tile's operands at a time: the registers are tight
            if constexpr (kTT > 1) __builtin_amdgcn_sched_barrier(0);
            const i32x8_t w8 = join8(w[i][r][0], w[i][r][1]);
            const Bf16Frag we = e4m3_to_bf16(w8);
#pragma unroll
            for (int t = 0; t < kTT; ++t) {
              f32x4_t d;
              if constexpr (kHold) {
                d = mfma_exact_block(we, xe[t]);
              } else {
                i32x8_t v = x8[t];
                asm volatile("" : "+v"(v));  // converted here, not once for all row tiles
                d = mfma_exact_block(we, e4m3_to_bf16(v));
                __builtin_amdgcn_sched_barrier(0);
              }
              acc[r][t][0] = __builtin_fmaf(d[0], s0[t], acc[r][t][0]);
              acc[r][t][1] = __builtin_fmaf(d[1], s0[t], acc[r][t][1]);
              acc[r][t][2] = __builtin_fmaf(d[2], s1[t], acc[r][t][2]);
              acc[r][t][3] = __builtin_fmaf(d[3], s1[t], acc[r][t][3]);
            }
          }
          if constexpr (kTT > 1) __builtin_amdgcn_sched_barrier(0);
          if (kb + kWaves * kRing < Kb) {
            load_w(i, kb + kWaves * kRing);
            load_x(i, kb + kWaves * kRing);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r) sums.v[wave][r][lane] = acc[r][t];
      __syncthreads();
      const int r = t0 + 16 * t + m16;
      if (r >= n) continue;
      f32x4_t v = sums.v[0][wave][lane];
#pragma unroll
      for (int u = 1; u < kWaves; ++u) v += sums.v[u][wave][lane];
      if constexpr (kDown) {
        const size_t row = shared ? static_cast<size_t>(a.r_max) + r : static_cast<size_t>(base) + r;
        const u32x2_t o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        *reinterpret_cast<u32x2_t*>(a.y + row * a.d + rb * 64 + wave * 16 + 4 * g) = o;
      } else {
        float* hf = (shared ? a.hshf : a.hf) + static_cast<size_t>(base + r) * I;
        float2 o;
        o.x = swiglu(v[0], v[2]);
        o.y = swiglu(v[1], v[3]);
        *reinterpret_cast<float2*>(hf + rb * 32 + wave * 8 + 2 * g) = o;
      }
    }
  }
}

// kItems > 0: rows quantised here, at most 16 of an expert and kItems (row, K block)
// pairs. launch_bounds: two workgroups a CU, three with few items (the 16-token
// form alone needs fewer registers).
template <bool kDown, int kItems>
__global__ __launch_bounds__(64 * kWaves, kItems > 0 && kItems <= kFewItems ? 3 : 2) void ffn_kernel(
    FfnArgs a, int shared_blocks, int blocks) {
  __shared__ union Lds {
    Sums sums;
    FusedRows<kItems> rows;
    __device__ Lds() {}
  } lds;
  // workgroups: the shared expert's weight blocks, then (expert slot, block)
  int b = blockIdx.x, el = 0;
  const bool shared = b < shared_blocks;
  int n = a.S;
  if (!shared) {
    b -= shared_blocks;
    const int slot = b / blocks;
    b -= slot * blocks;
    if (slot >= a.active[0]) return;
    el = a.active[1 + slot];
    n = min(a.counts[el], a.S);
  }
  if constexpr (kItems > 0) {
    ffn_block<1, kDown, kItems>(a, shared, el, b, n, lds.sums, lds.rows);
  } else {
    if (n <= 16)
      ffn_block<1, kDown, 0>(a, shared, el, b, n, lds.sums, lds.rows);
    else
      ffn_block<4, kDown, 0>(a, shared, el, b, n, lds.sums, lds.rows);
  }
}

// the SwiGLU rows of both kinds to e4m3: 8 lanes a (row, K block), the routed ones
// (rows in front of *used) first
__global__ __launch_bounds__(256) void quant_h_kernel(FfnArgs a, const int32_t* __restrict__ used) {
  int item = (blockIdx.x * 256 + threadIdx.x) >> 3;
  const int l8 = threadIdx.x & 7;
  const int routed = a.r_max * (a.I / kFp8Block);
  const bool shared = item >= routed;
  if (shared) item -= routed;
  const RowSet& set = shared ? a.hsh : a.h;
  const int K = shared ? a.Is : a.I, Kb = K / kFp8Block;
  if (Kb == 0) return;
  const int row = item / Kb, kb = item - row * Kb;
  if (row >= (shared ? a.S : min(*used, a.r_max))) return;
  Raw16<float> v;
  load16<float>(static_cast<const float*>(set.x) + static_cast<size_t>(row) * K,
                      kb * kFp8Block + l8 * 16, K, v);
  float scale;
  const u32x4_t q = quant16(v, scale);
  *reinterpret_cast<u32x4_t*>(const_cast<uint8_t*>(set.xq) + static_cast<size_t>(row) * K +
                              kb * kFp8Block + l8 * 16) = q;
  if (l8 == 0) const_cast<float*>(set.xs)[static_cast<size_t>(kb) * set.rows + row] = scale;
}

template <bool kDown>
void launch_step(const FfnArgs& a, int items, int shared_blocks, int blocks, hipStream_t stream) {
  const unsigned grid = shared_blocks + a.n_local * blocks;
  if (items == 0)
    ffn_kernel<kDown, 0><<<grid, 64 * kWaves, 0, stream>>>(a, shared_blocks, blocks);
  else if (items <= kFewItems)
    ffn_kernel<kDown, kFewItems><<<grid, 64 * kWaves, 0, stream>>>(a, shared_blocks, blocks);
  else
    ffn_kernel<kDown, kFusedItems><<<grid, 64 * kWaves, 0, stream>>>(a, shared_blocks, blocks);
}

// (row, K block) pairs an expert may have where its workgroups quantise them, else 0
int fused_items(int S, int K) {
  const int items = S * (K / kFp8Block);
  return S <= kFusedRows && items <= kFusedItems ? items : 0;
}

bool weight_shape(const moe_dims& m, int which, int& n, int& N, int& K) {
  const bool shared = which == MOE_WS13 || which == MOE_WS2;
  if (which < MOE_W13 || which > MOE_WS2 || (shared && m.shared_I == 0)) return false;
  const int I = shared ? m.shared_I : m.I;
  const bool up = which == MOE_W13 || which == MOE_WS13;
  n = shared ? 1 : m.n_local;
  N = up ? 2 * I : m.d;
  K = up ? m.d : I;
  return true;
}

// workspace: x rows and scales, then routed and shared SwiGLU rows (fp32, e4m3, scales)
struct FfnLayout {
  size_t xq, xs, hf, hshf, hq, hs, hshq, hshs, total;
};

FfnLayout ffn_layout(const moe_dims& m) {
  const size_t S = m.S, R = r_max(m), I = m.I, Is = m.shared_I, d = m.d;
  FfnLayout l;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t p = at;
    at += round_up(bytes, 256);
    return p;
  };
  l.xq = take(S * d);
  l.xs = take(S * (d / 128) * 4);
  l.hf = take(R * I * 4);
  l.hshf = take(S * Is * 4);
  l.hq = take(R * I);
  l.hs = take(R * (I / 128) * 4);
  l.hshq = take(S * Is);
  l.hshs = take(S * (Is / 128) * 4);
  l.total = at;
  return l;
}

}  // namespace
}  // namespace moeblk

using namespace moeblk;

extern "C" {

size_t moe_packed_fp8_expert_bytes(const moe_dims* dims, int which) {
  int n, N, K;
  if (check_dims(dims) || !weight_shape(*dims, which, n, N, K)) return 0;
  return n * fp8_packed_bytes(N, K);
}

int moe_pack_fp8_expert(const moe_dims* dims, int which, const void* q, const float* scales,
                        void* packed, hipStream_t stream) {
  const int rc = check_dims(dims);
  if (rc) return rc;
  int n, N, K;
  MOE_REQUIRE(weight_shape(*dims, which, n, N, K), MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(q && scales && packed, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(q) && aligned16(scales) && aligned16(packed), MOE_ERR_ALIGN);
  const bool up = which == MOE_W13 || which == MOE_WS13;
  launch_fp8_pack(q, scales, packed, n, N, K, up ? MOE_W13 : MOE_W2, stream);
  return launch_status();
}

size_t moe_fp8_ffn_workspace_bytes(const moe_dims* dims) {
  return check_dims(dims) ? 0 : ffn_layout(*dims).total;
}

int moe_fp8_expert_ffn(const moe_dims* dims, const void* x, const void* w13_packed,
                       const void* w2_packed, const int32_t* counts, const int32_t* offsets,
                       const int32_t* rows, const int32_t* active, const void* ws13_packed,
                       const void* ws2_packed, void* y, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  const int rc = check_dims(dims);
  if (rc) return rc;
  const moe_dims& m = *dims;
  const bool sh = m.shared_I > 0;
  MOE_REQUIRE(x && w13_packed && w2_packed && counts && offsets && rows && active && y && workspace,
              MOE_ERR_NULL);
  MOE_REQUIRE(!sh || (ws13_packed && ws2_packed), MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(x) && aligned16(w13_packed) && aligned16(w2_packed) && aligned16(counts) &&
                  aligned16(offsets) && aligned16(rows) && aligned16(active) &&
                  aligned16(ws13_packed) && aligned16(ws2_packed) && aligned16(y) &&
                  aligned16(workspace),
              MOE_ERR_ALIGN);
  const FfnLayout l = ffn_layout(m);
  MOE_REQUIRE(workspace_bytes >= l.total, MOE_ERR_WORKSPACE);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  const int R = r_max(m);
  FfnArgs a;
  a.S = m.S, a.d = m.d, a.n_local = m.n_local, a.r_max = R, a.I = m.I, a.Is = m.shared_I;
  a.counts = counts, a.offsets = offsets, a.rows = rows, a.active = active;
  a.w13 = static_cast<const uint8_t*>(w13_packed), a.w2 = static_cast<const uint8_t*>(w2_packed);
  a.ws13 = static_cast<const uint8_t*>(ws13_packed), a.ws2 = static_cast<const uint8_t*>(ws2_packed);
  a.x = RowSet{x, ws + l.xq, f32(l.xs), m.S};
  a.h = RowSet{f32(l.hf), ws + l.hq, f32(l.hs), R};
  a.hsh = RowSet{f32(l.hshf), ws + l.hshq, f32(l.hshs), m.S};
  a.hf = f32(l.hf), a.hshf = f32(l.hshf);
  a.y = static_cast<uint16_t*>(y);

  const int up_items = fused_items(m.S, m.d);
  if (!up_items) launch_fp8_quant(x, MOE_BF16, ws + l.xq, f32(l.xs), m.S, m.d, stream);
  launch_step<false>(a, up_items, m.shared_I / 32, m.I / 32, stream);
  const int down_items = fused_items(m.S, m.I > m.shared_I ? m.I : m.shared_I);
  if (!down_items) {
    const int items = R * (m.I / kFp8Block) + m.S * (m.shared_I / kFp8Block);
    quant_h_kernel<<<(items + 31) / 32, 256, 0, stream>>>(a, offsets + m.n_local);
  }
  launch_step<true>(a, down_items, sh ? m.d / 64 : 0, m.d / 64, stream);
  return launch_status();
}

}  // extern "C"
