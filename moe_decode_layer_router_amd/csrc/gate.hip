// gate.hip -- top-k of many rows' router logits with the routing weights, and
// the weights' gradient back to the logits (moe_gate, moe_gate_backward).
//
// With l the row's logits, P its picks and g the gradient of their weights:
//   sigmoid         w_s = s(l_s)                 dl_s = g_s w_s (1 - s(l_s))
//   sigmoid, renorm w_s = s(l_s) / sum_P s(l)    dl_s = w_s (1 - s(l_s)) (g_s - sum_P g w)
//   softmax         w_s = p_s over all experts   dl_e = p_e (sum of g over picks of e - sum_P g w)
//   softmax, renorm w_s = p_s over the picks     dl_s = w_s (g_s - sum_P g w)
// Scores are taken relative to the largest where that keeps them from vanishing:
// s(l) e^-m with m = min(max l, 0) is exp(min(l, 0) - m) / (1 + exp(-|l|)).
//
// Sixteen lanes hold a row (lanes16.h), four rows a wave. The forward takes the largest
// key in each of topk rounds, and lane s keeps pick s. Its rounds run on words of a key's
// upper 24 bits and the column (the lower one above), which all differ: a lane sorts its
// four largest, a round takes the largest of the 16 lanes' first ones and the lane that had it
// moves up (65536 x 256, topk 8: 750 vector instructions for four rows when each round went
// through all words, 529 so). Where the lower 8 bits could matter (a pick out of
// order with the next, or keys at the border that agree in 24 bits only) the wave takes
// the rounds on whole keys. The backward fills the row in LDS (zeros, or softmax's dense
// part), adds the picks' terms there and stores it whole.
#include <type_traits>

#include "common.h"
#include "host.h"
#include "lanes16.h"

namespace moeblk {
namespace {

constexpr int kGateRows = 16;  // rows a workgroup of 256 threads holds at a time
constexpr int kMaxE = 256;

constexpr float kLog2EHi = 1.44269504088896341f, kLog2ELo = 1.92596299112661746887e-8f;

// exp(x) to about an ulp: the argument's product with log2(e) in two parts (the
// hardware's exp2 alone is off by |x| 2^-24)
__device__ __forceinline__ float exp_near(float x) {
  const float t = x * kLog2EHi;
  const float r = __builtin_fmaf(x, kLog2ELo, __builtin_fmaf(x, kLog2EHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // an infinite or NaN argument has no second part
  return __builtin_fabsf(t) <= 1e30f ? __builtin_fmaf(e, r * 0.693147180559945309f, e) : e;
}

// An order of fp32 keys as integers: NaN above all (whatever its sign), then as
// floats (-0 = +0). -inf, which is never picked, comes last: kNever.
constexpr uint32_t kNever = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return f != f ? 0xffffffffu : k;
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t row_max_u(uint32_t v) {
  v = max(v, dpp_u<0xb1>(v));
  v = max(v, dpp_u<0x4e>(v));
  v = max(v, dpp_u<0x141>(v));
  return max(v, dpp_u<0x140>(v));
}
__device__ __forceinline__ uint32_t row_min_u(uint32_t v) {
  v = min(v, dpp_u<0xb1>(v));
  v = min(v, dpp_u<0x4e>(v));
  v = min(v, dpp_u<0x141>(v));
  return min(v, dpp_u<0x140>(v));
}

struct GateArgs {
  const float *logits, *bias;  // bias: only what steers the selection
  int32_t* ids;
  float* w;
  int T, E, topk, score, renorm;
};

// A row's largest logit (0 if there is none) and its sum of exp(l - m), the same bits for either
// kernel. An exponential's argument (l - m) log2(e) is rounded once, which takes |l - m| 2^-24 of
// its term, 3.4 2^-24 of the sum at most (256 terms: the weighted mean of |l - m| stays below 3.4).
// With the constant's first part alone all terms would be off to the same side. 65536 x 256, the
// forward in us and its weights' error in the 2-norm: 19.6, 5.7e-8; the first part alone 19.1, 6.3e-8;
// exp_near 20.8, 5.6e-8.
template <int kNI>
__device__ __forceinline__ void softmax_row(const Row<kNI>& l, float& m, float& total) {
  m = l.v[0];
#pragma unroll
  for (int i = 1; i < 4 * kNI; ++i) m = fmaxf(m, l.v[i]);
  m = row_max(m);
  m = m == -INFINITY ? 0.0f : m;
  total = 0.0f;
#pragma unroll
  for (int i = 0; i < 4 * kNI; ++i) {
    const float x = l.v[i] - m;
    total += __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2EHi, x * kLog2ELo));
  }
  total = row_sum(total);
}

// Lane s of a row: pick s's logit v (`on`: there is one). Its weight, and 1 -
// sigmoid (1 for softmax) for the gradient; m, total: of the whole row, where
// the weights are softmax's over all experts.
__device__ __forceinline__ float pick_weight(float v, bool on, int score, int renorm, float m,
                                             float total, float& slope) {
  float a;
  slope = 1.0f;
  if (score == MOE_SCORE_SIGMOID) {
    const float top = renorm ? row_max(on ? v : -INFINITY) : 0.0f;
    m = top == -INFINITY ? 0.0f : fminf(top, 0.0f);
    const float e = exp_near(-fabsf(v));
    a = exp_near(fminf(v, 0.0f) - m) / (1.0f + e);
    if (v != v) a = v;  // fminf drops a NaN
    slope = (v >= 0.0f ? e : 1.0f) / (1.0f + e);
    total = 1.0f;
  } else {
    if (renorm) {
      m = row_max(on ? v : -INFINITY);
      m = m == -INFINITY ? 0.0f : m;
    }
    a = exp_near(v - m);
  }
  a = on ? a : 0.0f;
  if (renorm) total = row_sum(a);
  return total == 0.0f ? 0.0f : a / total;
}

// the topk rounds on whole keys: the row's pick s in lane s, -1 where there is none
template <int kNI>
__device__ __forceinline__ int pick_exact(uint32_t (&key)[4 * kNI], int topk, int j) {
  int id = -1;
  for (int s = 0; s < topk; ++s) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < 4 * kNI; ++i) m = max(m, key[i]);
    m = row_max_u(m);
    uint32_t col = 0xffffu;  // lowest column with the maximum: 64 i + c ascends with the index
#pragma unroll
    for (int i = 4 * kNI - 1; i >= 0; --i)
      col = key[i] == m ? static_cast<uint32_t>((i >> 2) * 64 + (i & 3)) : col;
    const uint32_t e = row_min_u(col == 0xffffu ? col : col + 4 * j);
#pragma unroll
    for (int i = 0; i < 4 * kNI; ++i)
      key[i] = e == static_cast<uint32_t>((i >> 2) * 64 + 4 * j + (i & 3)) ? 0u : key[i];
    if (j == s) id = m <= kNever ? -1 : static_cast<int>(e);
  }
  return id;
}

__device__ __forceinline__ void descend(uint32_t& a, uint32_t& b) {
  const uint32_t t = max(a, b);
  b = min(a, b);
  a = t;
}
__device__ __forceinline__ void sort4(uint32_t (&v)[4]) {
  descend(v[0], v[1]);
  descend(v[2], v[3]);
  descend(v[0], v[2]);
  descend(v[1], v[3]);
  descend(v[1], v[2]);
}
// the four largest of a and b, all descending
__device__ __forceinline__ void merge4(uint32_t (&a)[4], const uint32_t (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = max(a[i], b[3 - i]);
  descend(a[0], a[2]);
  descend(a[1], a[3]);
  descend(a[0], a[1]);
  descend(a[2], a[3]);
}
// A lane's four largest words, or those below `below`, descending (0: no more)
template <int kNI, bool kBelow>
__device__ __forceinline__ void largest_words(const uint32_t (&key)[4 * kNI], int j, uint32_t below,
                                              uint32_t (&best)[4]) {
#pragma unroll
  for (int i = 0; i < kNI; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      w[c] = (key[4 * i + c] & 0xffffff00u) | (255u - (i * 64 + 4 * j + c));
      if (kBelow) w[c] = w[c] < below ? w[c] : 0u;
    }
    sort4(w);
    if (i > 0) {
      merge4(best, w);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) best[c] = w[c];
    }
  }
}

template <int kNI>
__global__ __launch_bounds__(256, 7) void gate_kernel(GateArgs a) {
  const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int E = a.E;
  // the lanes of a row stay together, and so do the four rows of a wave (those behind the
  // last row take the last one)
  const int row = blockIdx.x * kGateRows + group;
  const float* lrow = a.logits + static_cast<size_t>(min(row, a.T - 1)) * E;
  Row<kNI> l;
  load_row<kNI>(a.logits, min(row, a.T - 1), E, j, l);
  float top = 0.0f, total = 1.0f;
  if (a.score == MOE_SCORE_SOFTMAX && !a.renorm) softmax_row<kNI>(l, top, total);
  if (a.bias) {
    Row<kNI> bias;
    load_row<kNI>(a.bias, 0, E, j, bias);
#pragma unroll
    for (int i = 0; i < 4 * kNI; ++i) l.v[i] += bias.v[i];
  }
  uint32_t key[4 * kNI];
#pragma unroll
  for (int i = 0; i < 4 * kNI; ++i) key[i] = order_key(l.v[i]);
  uint32_t best[4];  // the lane's largest words, descending
  largest_words<kNI, false>(key, j, 0, best);
  // lane s: the word of rank s, up to rank topk (there are at least 64)
  uint32_t m = row_max_u(best[0]), mine = m;
  for (int s = 1; s <= a.topk; ++s) {
    const bool taken = best[0] == m;
#pragma unroll
    for (int c = 0; c < 4; ++c) best[c] = taken ? (c < 3 ? best[c + 1] : 0u) : best[c];
    // a lane that gave four may have more: all that are left are below m
    if (kNI > 1 && __any(best[0] == 0)) largest_words<kNI, true>(key, j, m, best);
    m = row_max_u(best[0]);
    if (j == s) mine = m;
  }
  int id = mine <= kNever ? -1 : 255 - static_cast<int>(mine & 255u);
  float v = id >= 0 ? lrow[id] : -INFINITY;
  {
    // the picks' whole keys have to descend, and behind the last pick all keys that share
    // its 24 bits have to be equal to it
    const uint32_t exact = id >= 0 ? order_key(a.bias ? v + a.bias[id] : v) : 0u;
    const uint32_t after = static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(exact), 0x101, 0xf, 0xf, true));  // lane + 1
    bool bad = j < a.topk && exact < after;
    const int first = threadIdx.x & 48;  // the row's lane 0
    const uint32_t last = __shfl(mine, first + a.topk - 1, kWave), edge = __shfl(mine, first + a.topk, kWave);
    const bool tie = last >> 8 == edge >> 8 && edge > kNever;
    if (__any(tie)) {
      const uint32_t whole = __shfl(exact, first + a.topk - 1, kWave);
#pragma unroll
      for (int i = 0; i < 4 * kNI; ++i) bad = bad || (tie && key[i] >> 8 == last >> 8 && key[i] != whole);
    }
    if (__any(bad)) {
      id = pick_exact<kNI>(key, a.topk, j);
      v = id >= 0 ? lrow[id] : -INFINITY;
    }
  }
  const bool on = id >= 0 && j < a.topk;
  float slope;
  const float w = pick_weight(v, on, a.score, a.renorm, top, total, slope);
  if (j < a.topk && row < a.T) {
    const size_t at = static_cast<size_t>(row) * a.topk + j;
    a.ids[at] = id;
    a.w[at] = w;
  }
}

// LDS that lanes of one wave hand to each other: its accesses stay in order, in the
// code as well
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct GateBackwardArgs {
  const float* logits;
  const int32_t* ids;
  const float *dw, *dadd;
  float* dlogits;
  int T, E, topk, score, renorm;
};

template <int kNI, bool kDense>
__global__ __launch_bounds__(256) void gate_backward_kernel(GateBackwardArgs a) {
  __shared__ __attribute__((aligned(16))) float rows[kGateRows][64 * kNI];
  const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int E = a.E, row = blockIdx.x * kGateRows + group;
  float* mine = rows[group];
  int id = -1;
  float dw = 0.0f;
  if (row < a.T && j < a.topk) {
    id = a.ids[static_cast<size_t>(row) * a.topk + j];
    dw = a.dw[static_cast<size_t>(row) * a.topk + j];
  }
  Row<kNI> l;
  if constexpr (kDense) load_row<kNI>(a.logits, min(row, a.T - 1), E, j, l);
  const bool in = row < a.T, on = id >= 0 && id < E;
  const float v = on ? a.logits[static_cast<size_t>(row) * E + id] : -INFINITY;
  float m = 0.0f, total = 1.0f;
  if constexpr (kDense) softmax_row<kNI>(l, m, total);
  float slope;
  const float w = pick_weight(v, on, a.score, a.renorm, m, total, slope);
  const float g = on ? dw : 0.0f;
  const float mean = kDense || a.renorm ? row_sum(on ? g * w : 0.0f) : 0.0f;
  // the row in LDS: its 16 lanes are of one wave
#pragma unroll
  for (int i = 0; i < kNI; ++i) {
    f32x4_t q = {0, 0, 0, 0};
    if constexpr (kDense) {
      const float scale = total == 0.0f ? 0.0f : -mean / total;
#pragma unroll
      for (int c = 0; c < 4; ++c) q[c] = exp_near(l.v[4 * i + c] - m) * scale;
    }
    *reinterpret_cast<f32x4_t*>(mine + 64 * i + 4 * j) = q;
  }
  wave_sync();
  if (on) atomicAdd(&mine[id], kDense ? w * g : w * slope * (g - mean));  // the same id twice adds up
  wave_sync();
  if (in) {
    const size_t at = static_cast<size_t>(row) * E;
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      const int e = 64 * i + 4 * j;
      f32x4_t q = *reinterpret_cast<const f32x4_t*>(mine + e);
      if (e + 4 <= E) {
        if (a.dadd) q += *reinterpret_cast<const f32x4_any_t*>(a.dadd + at + e);
        __builtin_nontemporal_store(q, reinterpret_cast<f32x4_any_t*>(a.dlogits + at + e));
      } else {
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (e + c < E) a.dlogits[at + e + c] = a.dadd ? q[c] + a.dadd[at + e + c] : q[c];
      }
    }
  }
}

// A workgroup a kGateRows rows, no loop: the scheduler keeps some waves loading while others
// compute. 2048 workgroups in a loop, the next rows' loads ahead: 65536 x 256 27 and 25 us in place of
// 19 and 21 (floors 14 and 26 at a copy's 5.1 TB/s: the gradient's stores pass the caches, with
// which they took 2 us longer). The forward is bound by its vector instructions, 14 us of them.
inline unsigned gate_grid(int T) { return static_cast<unsigned>((T + kGateRows - 1) / kGateRows); }

template <typename F>
void for_width(int E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>());
  else if (E <= 128) f(std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 4>());
}

}  // namespace

int check_gate_dims(const moe_gate_dims* d) {
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL);
  MOE_REQUIRE(d->T >= 1 && d->T <= 1 << 22, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->E >= 1 && d->E <= kMaxE, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->topk >= 1 && d->topk <= 8 && d->topk <= d->E, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->score == MOE_SCORE_SIGMOID || d->score == MOE_SCORE_SOFTMAX, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(d->renorm == 0 || d->renorm == 1, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(d->bias_mode == 0 || d->bias_mode == 1, MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

}  // namespace moeblk

using namespace moeblk;

extern "C" {

int moe_check_gate_dims(const moe_gate_dims* dims) { return check_gate_dims(dims); }

int moe_gate(const moe_gate_dims* dims, const float* logits, const float* bias, int32_t* topk_ids,
             float* topk_w, hipStream_t stream) {
  const int rc = check_gate_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(logits && topk_ids && topk_w, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(logits) && aligned16(bias) && aligned16(topk_ids) && aligned16(topk_w),
              MOE_ERR_ALIGN);
  const GateArgs a = {logits,  dims->bias_mode == 1 ? bias : nullptr, topk_ids, topk_w,
                      dims->T, dims->E, dims->topk, dims->score, dims->renorm};
  for_width(dims->E, [&](auto ni) {
    gate_kernel<decltype(ni)::value><<<gate_grid(dims->T), 256, 0, stream>>>(a);
  });
  return launch_status();
}

int moe_gate_backward(const moe_gate_dims* dims, const float* logits, const int32_t* topk_ids,
                      const float* dtopk_w, const float* dadd, float* dlogits,
                      hipStream_t stream) {
  const int rc = check_gate_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(logits && topk_ids && dtopk_w && dlogits, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(logits) && aligned16(topk_ids) && aligned16(dtopk_w) && aligned16(dadd) &&
                  aligned16(dlogits),
              MOE_ERR_ALIGN);
  const GateBackwardArgs a = {logits,  topk_ids, dtopk_w,    dadd,        dlogits,
                              dims->T, dims->E,  dims->topk, dims->score, dims->renorm};
  const bool dense = dims->score == MOE_SCORE_SOFTMAX && !dims->renorm;
  for_width(dims->E, [&](auto ni) {
    constexpr int kNI = decltype(ni)::value;
    if (dense)
      gate_backward_kernel<kNI, true><<<gate_grid(dims->T), 256, 0, stream>>>(a);
    else
      gate_backward_kernel<kNI, false><<<gate_grid(dims->T), 256, 0, stream>>>(a);
  });
  return launch_status();
}

}  // extern "C"
