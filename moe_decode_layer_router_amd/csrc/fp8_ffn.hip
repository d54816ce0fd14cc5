// fp8_ffn.hip -- the expert FFNs on FP8 weights with block-128 scales
// (moe_fp8_expert_ffn), and their weight packing.
//
// Four launches: the rows x to e4m3; gate_up + SwiGLU of every (expert, block of
// 64 packed rows = 32 intermediates), h in fp32; h to e4m3; down of every
// (expert, 64 output rows). A workgroup's 8 waves take every eighth K block and
// stream the packed weights straight into registers.
#include "fp8_dev.h"
#include "fp8_launch.h"
#include "host.h"

namespace moeblk {
namespace {

constexpr int kWaves = 8;

struct RowSet {
  const uint8_t* xq;  // e4m3 rows
  const float* xs;    // scales [Kb][xs_rows]
  int xs_rows;        // rows of the scale array
  size_t Kp;          // bytes a row
};

// 64 packed weight rows x 16 kTT tokens over all K blocks: acc[r][t] of this
// wave. `tok`: this lane's row of the row set for each token tile. Lane rows 0,
// 1 of a D tile take the scale sw0, rows 2, 3 sw1 (gate / up; the same array for
// down).
template <int kTT>
__device__ __forceinline__ void stream_rows(const uint8_t* wt, const float* sw0, const float* sw1,
                                            int Kb, const RowSet& x, const int (&tok)[kTT],
                                            int wave, int lane, f32x4_t (&acc)[4][kTT]) {
  const int g = lane >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < kTT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
  for (int kb = wave; kb < Kb; kb += kWaves) {
    Bf16Frag a[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* p = wt + (static_cast<size_t>(r) * Kb + kb) * kFp8TileBytes + lane * 16;
      a[r] = e4m3_to_bf16(join8(ld_nt<u32x4_t>(p), ld_nt<u32x4_t>(p + 1024)));
    }
    const float w0 = sw0[kb], w1 = sw1[kb];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const uint8_t* p = x.xq + tok[t] * x.Kp + kb * kFp8Block + 32 * g;
      const Bf16Frag b = e4m3_to_bf16(join8(*reinterpret_cast<const u32x4_t*>(p),
                                            *reinterpret_cast<const u32x4_t*>(p + 16)));
      const float s = x.xs[static_cast<size_t>(kb) * x.xs_rows + tok[t]];
      const float s0 = s * w0, s1 = s * w1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f32x4_t d = mfma_exact_block(a[r], b);
        acc[r][t][0] = __builtin_fmaf(d[0], s0, acc[r][t][0]);
        acc[r][t][1] = __builtin_fmaf(d[1], s0, acc[r][t][1]);
        acc[r][t][2] = __builtin_fmaf(d[2], s1, acc[r][t][2]);
        acc[r][t][3] = __builtin_fmaf(d[3], s1, acc[r][t][3]);
      }
    }
  }
}

// sums the waves' acc[.][t] in wave order; wave r < 4 returns the sum of row
// tile r in its lanes
template <int kTT>
__device__ __forceinline__ f32x4_t sum_waves(f32x4_t (&red)[kWaves][4][64],
                                             const f32x4_t (&acc)[4][kTT], int t, int wave,
                                             int lane) {
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 4; ++r) red[wave][r][lane] = acc[r][t];
  __syncthreads();
  f32x4_t s = {0, 0, 0, 0};
  if (wave < 4) {
    s = red[0][wave][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) s += red[v][wave][lane];
  }
  return s;
}

struct FfnArgs {
  int S, d, n_local, r_max, I, Is;
  const int32_t *counts, *offsets, *rows, *active;
  const uint8_t *w13, *w2, *ws13, *ws2;  // packed; ws*: shared expert or NULL
  RowSet x;                              // quantised input rows
  RowSet h, hsh;                         // quantised SwiGLU rows: routed, shared
  float *hf, *hshf;                      // fp32 SwiGLU rows: routed [r_max][I], shared [S][Is]
  uint16_t* y;
};

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// token groups of one weight block, 16 kTT tokens each
template <int kTT, bool kDown>
__device__ __forceinline__ void ffn_block(const FfnArgs& a, bool shared, int el, int rb,
                                          f32x4_t (&red)[kWaves][4][64]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m16 = lane & 15, g = lane >> 4;
  const int I = shared ? a.Is : a.I;
  const int N = kDown ? a.d : 2 * I, K = kDown ? I : a.d, Kb = K / kFp8Block;
  const uint8_t* w = kDown ? (shared ? a.ws2 : a.w2) : (shared ? a.ws13 : a.w13);
  w += el * fp8_packed_bytes(N, K);
  const float* sc = reinterpret_cast<const float*>(w + fp8_tile_bytes(N, K));
  const uint8_t* wt = w + static_cast<size_t>(rb) * 4 * Kb * kFp8TileBytes;
  const float* sw0 = sc + static_cast<size_t>(kDown ? rb / 2 : rb / 4) * Kb;
  const float* sw1 = kDown ? sw0 : sc + static_cast<size_t>((I / 128 + rb / 4)) * Kb;
  const int base = shared ? 0 : a.offsets[el];
  const int n = shared ? a.S : a.counts[el];
  const RowSet x = kDown ? (shared ? a.hsh : a.h) : a.x;
  for (int t0 = 0; t0 < n; t0 += 16 * kTT) {
    int tok[kTT];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const int r = min(t0 + 16 * t + m16, n - 1);
      tok[t] = (kDown || shared) ? base + r : min(max(a.rows[base + r], 0), a.S - 1);
    }
    f32x4_t acc[4][kTT];
    stream_rows<kTT>(wt, sw0, sw1, Kb, x, tok, wave, lane, acc);
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
      const f32x4_t s = sum_waves<kTT>(red, acc, t, wave, lane);
      const int r = t0 + 16 * t + m16;
      if (wave >= 4 || r >= n) continue;
      if constexpr (kDown) {
        const size_t row = shared ? static_cast<size_t>(a.r_max) + r : static_cast<size_t>(base) + r;
        const u32x2_t v = {pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        *reinterpret_cast<u32x2_t*>(a.y + row * a.d + rb * 64 + wave * 16 + 4 * g) = v;
      } else {
        float* hf = (shared ? a.hshf : a.hf) + static_cast<size_t>(base + r) * I;
        float2 v;
        v.x = swiglu(s[0], s[2]);
        v.y = swiglu(s[1], s[3]);
        *reinterpret_cast<float2*>(hf + rb * 32 + wave * 8 + 2 * g) = v;
      }
    }
  }
}

// workgroups: the shared expert's weight blocks, then (expert slot, block)
template <bool kDown>
__global__ __launch_bounds__(512) void ffn_kernel(FfnArgs a, int shared_blocks, int blocks) {
  __shared__ f32x4_t red[kWaves][4][64];
  int b = blockIdx.x, el = 0;
  const bool shared = b < shared_blocks;
  int n = a.S;
  if (!shared) {
    b -= shared_blocks;
    const int slot = b / blocks;
    b -= slot * blocks;
    if (slot >= a.active[0]) return;
    el = a.active[1 + slot];
    n = a.counts[el];
  }
  if (n <= 16)
    ffn_block<1, kDown>(a, shared, el, b, red);
  else if (n <= 32)
    ffn_block<2, kDown>(a, shared, el, b, red);
  else
    ffn_block<4, kDown>(a, shared, el, b, red);
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
  l.total = at + 256;
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
  a.x = RowSet{ws + l.xq, f32(l.xs), m.S, static_cast<size_t>(m.d)};
  a.h = RowSet{ws + l.hq, f32(l.hs), R, static_cast<size_t>(m.I)};
  a.hsh = RowSet{ws + l.hshq, f32(l.hshs), m.S, static_cast<size_t>(m.shared_I)};
  a.hf = f32(l.hf), a.hshf = f32(l.hshf);
  a.y = static_cast<uint16_t*>(y);

  launch_fp8_quant(x, MOE_BF16, ws + l.xq, f32(l.xs), m.S, m.d, nullptr, stream);
  const int up_sh = m.shared_I / 32, up = m.I / 32;
  ffn_kernel<false><<<up_sh + m.n_local * up, 512, 0, stream>>>(a, up_sh, up);
  launch_fp8_quant(a.hf, MOE_FP32, ws + l.hq, f32(l.hs), R, m.I, offsets + m.n_local, stream);
  if (sh) launch_fp8_quant(a.hshf, MOE_FP32, ws + l.hshq, f32(l.hshs), m.S, m.shared_I, nullptr, stream);
  const int dn = m.d / 64, dn_sh = sh ? dn : 0;
  ffn_kernel<true><<<dn_sh + m.n_local * dn, 512, 0, stream>>>(a, dn_sh, dn);
  return launch_status();
}

}  // extern "C"
