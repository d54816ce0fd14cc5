// balance.hip -- per-expert counts of the picks, the router's balance loss and
// its gradient (moe_expert_counts, moe_balance_loss, moe_balance_backward).
//
// With p the token's normalised scores, c[b][e] the picks of expert e in
// sequence b (T_b rows) and P[b][e] the mean of p over its rows,
//   L = coef / B * sum_b sum_e E / (topk T_b) c[b][e] P[b][e].
// The counts are constants for the gradient: with a[e] = g coef / B E / (topk
// T_b^2) c[b][e],
//   dL/dl_j = p_j (1 - s_j) (a_j - sum_e a_e p_e)   (sigmoid scores s)
//   dL/dl_j = p_j (a_j - sum_e a_e p_e)             (softmax).
// Forward is bound by reading the logits once, backward by reading and writing
// them once. A workgroup of the forward takes kChunk rows; where a chunk c meets
// a sequence b it leaves its sums in slot c + b (walking the rows, either index
// grows from one meeting to the next, so slots do not collide and there are at
// most chunks + sequences of them). A second launch sums each sequence's slots
// in chunk order in fp64: no result depends on an order of atomics.
#include <math.h>

#include "common.h"
#include "host.h"

namespace moeblk {
namespace {

constexpr int kChunk = 64;  // rows a forward workgroup takes
constexpr int kMaxE = 256;
constexpr int kPer = kMaxE / kWave;  // logits a lane holds: columns lane + 64 i

__device__ __forceinline__ int seq_start(const int32_t* starts, int b, int T) {
  if (!starts) return b == 0 ? 0 : T;
  return min(max(starts[b], 0), T);
}

// the last sequence that starts at or before `row` (0 if none does)
__device__ __forceinline__ int find_seq(const int32_t* starts, int n_seq, int row, int T) {
  if (!starts) return 0;
  int lo = 0, hi = n_seq;  // invariant: start(lo) <= row (or lo = 0), start(hi) > row (or hi = n_seq)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(starts, mid, T) <= row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}

// One row's normalised scores p of this lane's columns, and slope = dp_j/dl_j's
// factor p_j (1 - s_j) or p_j. Scores are taken relative to the row's largest
// where that keeps them from vanishing: sigmoid(l) e^{-m} with m = min(max l, 0)
// is exp(min(l, 0) - m) / (1 + exp(-|l|)). A row whose logits are all -inf has
// p = 0.
__device__ __forceinline__ void row_scores(const float (&l)[kPer], int score, float (&p)[kPer],
                                           float (&slope)[kPer]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) m = fmaxf(m, l[i]);
  m = wave_max(m);
  const bool none = m == -INFINITY;
  if (score == MOE_SCORE_SIGMOID) {
    m = none ? 0.0f : fminf(m, 0.0f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float e = expf(-fabsf(l[i]));
      const float r = 1.0f / (1.0f + e);
      const float num = m == 0.0f ? (l[i] >= 0.0f ? 1.0f : e) : expf(fminf(l[i], 0.0f) - m);
      p[i] = num * r;
      slope[i] = (l[i] >= 0.0f ? e : 1.0f) * r;  // 1 - sigmoid
    }
  } else {
    m = none ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      p[i] = expf(l[i] - m);
      slope[i] = 1.0f;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s += p[i];
  s = wave_sum(s);
  const float inv = none ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] *= inv;
    slope[i] *= p[i];
  }
}

__device__ __forceinline__ void load_row(const float* logits, size_t row, int E, int lane,
                                         float (&l)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + kWave * i;
    l[i] = e < E ? logits[row * E + e] : -INFINITY;
  }
}

// ---------------------------------------------------------------- forward

// logits NULL: counts only
__global__ __launch_bounds__(256) void chunk_kernel(const float* __restrict__ logits,
                                                    const int32_t* __restrict__ ids,
                                                    const int32_t* __restrict__ starts,
                                                    int32_t* __restrict__ slot_counts,
                                                    float* __restrict__ slot_probs, int T, int E,
                                                    int topk, int n_seq, int score) {
  __shared__ int cnt[kMaxE];
  __shared__ float sums[4][kMaxE];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = blockIdx.x;
  const int lo = c * kChunk, hi = min(T, lo + kChunk);
  int b = find_seq(starts, n_seq, lo, T);
  for (; b < n_seq; ++b) {
    const int s0 = max(lo, seq_start(starts, b, T)), s1 = min(hi, seq_start(starts, b + 1, T));
    if (s0 >= hi) break;
    if (s1 <= s0) continue;
    __syncthreads();
    cnt[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < (s1 - s0) * topk; i += 256) {
      const int e = ids[static_cast<size_t>(s0) * topk + i];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    if (logits) {
      float acc[kPer] = {};
      for (int row = s0 + wave; row < s1; row += 4) {
        float l[kPer], p[kPer], slope[kPer];
        load_row(logits, row, E, lane, l);
        row_scores(l, score, p, slope);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += p[i];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) sums[wave][lane + kWave * i] = acc[i];
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e < E) {
      const size_t at = static_cast<size_t>(c + b) * E + e;
      slot_counts[at] = cnt[e];
      if (logits) slot_probs[at] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
    }
  }
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// workgroup (b, 64 experts): wave v sums the slots v, v + 4, ... of its
// sequence's chunks. The last workgroup to finish adds the terms of the loss.
__global__ __launch_bounds__(256) void reduce_kernel(const int32_t* __restrict__ slot_counts,
                                                     const float* __restrict__ slot_probs,
                                                     const int32_t* __restrict__ starts,
                                                     int32_t* __restrict__ counts,
                                                     float* __restrict__ probs,
                                                     float* __restrict__ loss, double* terms,
                                                     int32_t* done, int T, int E, int topk,
                                                     int n_seq, float coef) {
  __shared__ int cnt[4][kWave];
  __shared__ double sums[4][kWave];
  __shared__ int last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int groups = (E + kWave - 1) / kWave;
  const int b = blockIdx.x / groups, e = (blockIdx.x % groups) * kWave + lane;
  const int s0 = seq_start(starts, b, T), s1 = seq_start(starts, b + 1, T);
  int n = 0;
  double p = 0.0;
  if (s1 > s0 && e < E) {
    for (int c = s0 / kChunk + wave; c <= (s1 - 1) / kChunk; c += 4) {
      const size_t at = static_cast<size_t>(c + b) * E + e;
      n += slot_counts[at];
      if (loss) p += slot_probs[at];
    }
  }
  cnt[wave][lane] = n;
  sums[wave][lane] = p;
  __syncthreads();
  double term = 0.0;
  if (wave == 0) {
    n = cnt[0][lane] + cnt[1][lane] + cnt[2][lane] + cnt[3][lane];
    p = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
    const double rows = s1 > s0 ? s1 - s0 : 1;
    p /= rows;
    if (e < E) {
      counts[static_cast<size_t>(b) * E + e] = n;
      if (loss) probs[static_cast<size_t>(b) * E + e] = static_cast<float>(p);
      term = static_cast<double>(E) / (topk * rows) * n * p;
    }
    term = wave_sum_f64(term);
  }
  if (!loss) return;
  if (threadIdx.x == 0) {
    __hip_atomic_store(&terms[blockIdx.x], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __threadfence();
    last = __hip_atomic_fetch_add(done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last || wave != 0) return;
  double sum = 0.0;
  for (unsigned i = lane; i < gridDim.x; i += kWave)
    sum += __hip_atomic_load(&terms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = wave_sum_f64(sum);
  if (lane == 0) {
    *loss = static_cast<float>(sum * static_cast<double>(coef) / n_seq);
    __hip_atomic_store(done, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// ---------------------------------------------------------------- backward

__global__ __launch_bounds__(256) void backward_kernel(const float* __restrict__ logits,
                                                       const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ starts,
                                                       const float* __restrict__ dloss,
                                                       float* __restrict__ dlogits, int T, int E,
                                                       int topk, int n_seq, float coef,
                                                       int score) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int lo = blockIdx.x * kChunk, hi = min(T, lo + kChunk);
  const float g = dloss ? *dloss : 1.0f;
  int b = find_seq(starts, n_seq, lo, T);
  for (; b < n_seq; ++b) {
    const int q0 = seq_start(starts, b, T), q1 = seq_start(starts, b + 1, T);
    const int s0 = max(lo, q0), s1 = min(hi, q1);
    if (s0 >= hi) break;
    if (s1 <= s0) continue;
    const double rows = q1 - q0;
    const float f = static_cast<float>(static_cast<double>(g) * coef / n_seq * E /
                                       (topk * rows * rows));
    float a[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + kWave * i;
      a[i] = e < E ? f * static_cast<float>(counts[static_cast<size_t>(b) * E + e]) : 0.0f;
    }
    for (int row = s0 + wave; row < s1; row += 4) {
      float l[kPer], p[kPer], slope[kPer];
      load_row(logits, row, E, lane, l);
      row_scores(l, score, p, slope);
      float mean = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mean = __builtin_fmaf(a[i], p[i], mean);
      mean = wave_sum(mean);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + kWave * i;
        if (e < E) dlogits[static_cast<size_t>(row) * E + e] = slope[i] * (a[i] - mean);
      }
    }
  }
}

int check_balance_dims(const moe_balance_dims* d) {
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL);
  MOE_REQUIRE(d->T >= 1 && d->T <= (1 << 22), MOE_ERR_SHAPE);
  MOE_REQUIRE(d->E >= 1 && d->E <= kMaxE, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->topk >= 1 && d->topk <= 8 && d->topk <= d->E, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->n_seq >= 1 && d->n_seq <= 4096, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->score == MOE_SCORE_SIGMOID || d->score == MOE_SCORE_SOFTMAX, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(isfinite(d->coef), MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

inline int chunks(const moe_balance_dims& d) { return (d.T + kChunk - 1) / kChunk; }
inline int reduce_groups(const moe_balance_dims& d) { return d.n_seq * ((d.E + 63) / 64); }

// workspace: the done counter (zero between calls), the loss terms, the slots
struct BalanceLayout {
  size_t terms, counts, probs, total;
};

BalanceLayout balance_layout(const moe_balance_dims& d) {
  BalanceLayout l;
  const size_t slots = static_cast<size_t>(chunks(d) + d.n_seq) * d.E;
  l.terms = 256;
  l.counts = l.terms + round_up(static_cast<size_t>(reduce_groups(d)) * 8, 256);
  l.probs = l.counts + round_up(slots * 4, 256);
  l.total = l.probs + round_up(slots * 4, 256);
  return l;
}

int forward(const moe_balance_dims* dims, const float* logits, const int32_t* topk_ids,
            const int32_t* seq_starts, int32_t* counts, float* probs, float* loss, void* workspace,
            size_t workspace_bytes, hipStream_t stream) {
  const moe_balance_dims& m = *dims;
  MOE_REQUIRE(topk_ids && counts && workspace && (seq_starts || m.n_seq == 1), MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(topk_ids) && aligned16(seq_starts) && aligned16(counts) &&
                  aligned16(workspace),
              MOE_ERR_ALIGN);
  const BalanceLayout l = balance_layout(m);
  MOE_REQUIRE(workspace_bytes >= l.total, MOE_ERR_WORKSPACE);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* sc = reinterpret_cast<int32_t*>(ws + l.counts);
  float* sp = reinterpret_cast<float*>(ws + l.probs);
  chunk_kernel<<<chunks(m), 256, 0, stream>>>(logits, topk_ids, seq_starts, sc, sp, m.T, m.E,
                                              m.topk, m.n_seq, m.score);
  reduce_kernel<<<reduce_groups(m), 256, 0, stream>>>(
      sc, sp, seq_starts, counts, probs, loss, reinterpret_cast<double*>(ws + l.terms),
      reinterpret_cast<int32_t*>(ws), m.T, m.E, m.topk, m.n_seq, m.coef);
  return launch_status();
}

}  // namespace
}  // namespace moeblk

using namespace moeblk;

extern "C" {

int moe_check_balance_dims(const moe_balance_dims* dims) { return check_balance_dims(dims); }

size_t moe_balance_workspace_bytes(const moe_balance_dims* dims) {
  return check_balance_dims(dims) ? 0 : balance_layout(*dims).total;
}

int moe_expert_counts(const moe_balance_dims* dims, const int32_t* topk_ids,
                      const int32_t* seq_starts, int32_t* counts, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_balance_dims(dims);
  if (rc) return rc;
  return forward(dims, nullptr, topk_ids, seq_starts, counts, nullptr, nullptr, workspace,
                 workspace_bytes, stream);
}

int moe_balance_loss(const moe_balance_dims* dims, const float* logits, const int32_t* topk_ids,
                     const int32_t* seq_starts, int32_t* counts, float* probs, float* loss,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = check_balance_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(logits && probs && loss, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(logits) && aligned16(probs) && aligned16(loss), MOE_ERR_ALIGN);
  return forward(dims, logits, topk_ids, seq_starts, counts, probs, loss, workspace,
                 workspace_bytes, stream);
}

int moe_balance_backward(const moe_balance_dims* dims, const float* logits, const int32_t* counts,
                         const int32_t* seq_starts, const float* dloss, float* dlogits,
                         hipStream_t stream) {
  const int rc = check_balance_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(logits && counts && dlogits && (seq_starts || dims->n_seq == 1), MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(logits) && aligned16(counts) && aligned16(seq_starts) &&
                  aligned16(dloss) && aligned16(dlogits),
              MOE_ERR_ALIGN);
  backward_kernel<<<chunks(*dims), 256, 0, stream>>>(logits, counts, seq_starts, dloss, dlogits,
                                                     dims->T, dims->E, dims->topk, dims->n_seq,
                                                     dims->coef, dims->score);
  return launch_status();
}

}  // extern "C"
