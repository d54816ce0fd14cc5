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
// them once. Sixteen lanes hold a row (four rows a wave): its maximum and sums
// are four steps within a DPP row, no LDS.
//
// A workgroup of the forward takes a chunk of rows; where a chunk c meets a
// sequence b it leaves its sums in slot c + b (walking the rows, either index
// grows from one meeting to the next, so slots do not collide and there are at
// most chunks + sequences of them). A second launch sums each sequence's slots
// in a fixed order in fp64: no result depends on an order of atomics. With few
// slots (up to 16: T <= 240 in one sequence) the last workgroup of the first launch
// does that instead, which saves a launch of about 3 us.
//
// T = 65536, E = 256: forward 19.2 us (3.6 TB/s) and 7.5 for the second launch, gradient
// 27.8 us (4.8 TB/s); T = 128: 7.2 and 6.3 us. Sigmoid scores take 2.5 and 4 us more than
// softmax's; the counts alone 8.6 us (65536 rows of 8) and 4.6.
#include <math.h>

#include "common.h"
#include "host.h"
#include "lanes16.h"

namespace moeblk {
namespace {

constexpr int kMaxE = 256;
constexpr int kPass = 16;      // rows a workgroup of 256 threads holds at a time
constexpr int kOneSlots = 16;  // most slots the last workgroup of the first launch sums

// Rows a workgroup takes: at least a pass, about 1024 (forward) or 2048 (backward:
// no sums to hand over) workgroups, at most 256 rows (fp32 sums over a chunk).
__host__ __device__ inline int chunk_rows(int T, int groups) {
  const int per = (T + groups - 1) / groups;
  const int r = (per + kPass - 1) / kPass * kPass;
  return r > 256 ? 256 : r;
}
__host__ __device__ inline int forward_rows(int T) { return chunk_rows(T, 1024); }
__host__ __device__ inline int backward_rows(int T) { return chunk_rows(T, 2048); }

__device__ __forceinline__ int seq_start(const int32_t* starts, int b, int T) {
  if (!starts) return b == 0 ? 0 : T;
  return min(max(starts[b], 0), T);
}

// The starts as a wave sees them: up to 63 sequences lie in its lanes (one load,
// no dependent search), more are searched in memory.
struct Starts {
  const int32_t* p;
  int n_seq, T, mine;
  __device__ Starts(const int32_t* starts, int n, int rows) : p(starts), n_seq(n), T(rows), mine(0) {
    if (n < kWave) mine = seq_start(p, min(static_cast<int>(threadIdx.x & (kWave - 1)), n), T);
  }
  __device__ int at(int b) const {  // b: the same in all lanes
    if (n_seq < kWave) return __builtin_amdgcn_readlane(mine, b);
    return seq_start(p, b, T);
  }
  // the last sequence that starts at or before `row` (0 if none does)
  __device__ int find(int row) const {
    if (n_seq < kWave) {
      const uint64_t m = __ballot(mine <= row && static_cast<int>(threadIdx.x & (kWave - 1)) < n_seq);
      return m ? 63 - __builtin_clzll(m) : 0;
    }
    int lo = 0, hi = n_seq;  // start(lo) <= row (or lo = 0), start(hi) > row (or hi = n_seq)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seq_start(p, mid, T) <= row)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
};

// One row's normalised scores p of this lane's columns, and slope = p_j (1 -
// s_j) or p_j (kSlope). Scores are taken relative to the row's largest where
// that keeps them from vanishing: sigmoid(l) e^{-m} with m = min(max l, 0) is
// exp(min(l, 0) - m) / (1 + exp(-|l|)). A row whose logits are all -inf has
// p = 0.
template <int kNI, bool kSlope>
__device__ __forceinline__ void row_scores(const Row<kNI>& l, int score, Row<kNI>& p,
                                           Row<kNI>& slope) {
  constexpr int n = 4 * kNI;
  float m = l.v[0];
#pragma unroll
  for (int i = 1; i < n; ++i) m = fmaxf(m, l.v[i]);
  m = row_max(m);
  const bool none = m == -INFINITY;
  if (score == MOE_SCORE_SIGMOID) {
    m = none ? 0.0f : fminf(m, 0.0f);
    const bool low = __any(m < 0.0f);  // a row of this wave has no logit above zero
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float x = l.v[i];
      const float e = exp_hw(-fabsf(x));
      const float r = __builtin_amdgcn_rcpf(1.0f + e);
      float num = x >= 0.0f ? 1.0f : e;
      if (low) num = m < 0.0f ? exp_hw(fminf(x, 0.0f) - m) : num;
      p.v[i] = num * r;
      if constexpr (kSlope) slope.v[i] = (x >= 0.0f ? e : 1.0f) * r;  // 1 - sigmoid
      if (x != x) p.v[i] = x;
    }
  } else {
    m = none ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      p.v[i] = exp_hw(l.v[i] - m);
      if constexpr (kSlope) slope.v[i] = 1.0f;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < n; ++i) s += p.v[i];
  s = row_sum(s);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;  // zero only where all are -inf; NaN stays
#pragma unroll
  for (int i = 0; i < n; ++i) {
    p.v[i] *= inv;
    if constexpr (kSlope) slope.v[i] *= p.v[i];
  }
}

// ---------------------------------------------------------------- forward

struct ForwardArgs {
  const float* logits;  // NULL: counts only
  const int32_t *ids, *starts;
  int32_t* slot_counts;
  float* slot_probs;
  int32_t* counts;
  float *probs, *loss;
  double* terms;
  int32_t* done;  // zero between calls
  int T, E, topk, n_seq, score;
  float coef;
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

template <typename T>
__device__ __forceinline__ void store_through(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T load_through(const T* p) {
  return __hip_atomic_load(const_cast<T*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Counts this workgroup as done; true in all threads of the last one (which
// sets the counter back). What the others stored through before is visible to its
// load_through: each thread waits for its own stores first.
__device__ __forceinline__ bool last_workgroup(int32_t* done) {
  __shared__ int last;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) {
    last = __hip_atomic_fetch_add(done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           static_cast<int>(gridDim.x) - 1;
    if (last) __hip_atomic_store(done, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return last;
}

// The sums of (b, kJ experts) over the sequence's slots by kReduce threads: expert
// tid % kJ, every kReduce / kJ-th slot (1024 threads against 256: one sequence of 65536
// rows, 1024 slots, 75 -> 60 us with the gradient). Returns the kJ experts' loss term in thread 0.
constexpr int kReduce = 1024;

template <int kJ>
__device__ __forceinline__ double reduce_group(const ForwardArgs& a, int b, int e0) {
  constexpr int kWaves = kReduce / kWave;
  __shared__ int cnt[kWaves][kJ + 1];
  __shared__ double sums[kWaves][kJ + 1];
  const int j = threadIdx.x % kJ, k = threadIdx.x / kJ, wave = threadIdx.x / kWave;
  const int e = e0 + j;
  const int rows = forward_rows(a.T);
  const int s0 = seq_start(a.starts, b, a.T), s1 = seq_start(a.starts, b + 1, a.T);
  int n = 0;
  double p = 0.0;
  if (s1 > s0 && e < a.E) {
    const int last = (s1 - 1) / rows;
#pragma unroll 8
    for (int c = s0 / rows + k; c <= last; c += kReduce / kJ) {
      const size_t at = static_cast<size_t>(c + b) * a.E + e;
      n += a.slot_counts[at];
      if (a.loss) p += a.slot_probs[at];
    }
  }
  // the slots of a wave, then the waves
#pragma unroll
  for (int m = kJ; m < kWave; m <<= 1) {
    n += __shfl_xor(n, m, kWave);
    p += __shfl_xor(p, m, kWave);
  }
  __syncthreads();  // the sums in front have been read
  if (threadIdx.x % kWave < kJ) {
    cnt[wave][j] = n;
    sums[wave][j] = p;
  }
  __syncthreads();
  double term = 0.0;
  if (threadIdx.x < kJ) {
    n = 0;
    p = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      n += cnt[i][j];
      p += sums[i][j];
    }
    const double len = s1 > s0 ? s1 - s0 : 1;
    p /= len;
    if (e < a.E) {
      a.counts[static_cast<size_t>(b) * a.E + e] = n;
      if (a.loss) a.probs[static_cast<size_t>(b) * a.E + e] = static_cast<float>(p);
      term = static_cast<double>(a.E) / (a.topk * len) * n * p;
    }
#pragma unroll
    for (int m = kJ / 2; m >= 1; m >>= 1) term += __shfl_xor(term, m, kJ);
  }
  return term;
}

__device__ __forceinline__ void store_loss(const ForwardArgs& a, double sum) {
  *a.loss = static_cast<float>(sum * static_cast<double>(a.coef) / a.n_seq);
}

template <int kNI, bool kOne>
__global__ __launch_bounds__(256) void chunk_kernel(ForwardArgs a) {
  __shared__ int cnt[kMaxE];
  __shared__ float sums[kPass][kMaxE];
  const int tid = threadIdx.x, j = tid & 15, group = tid >> 4;
  const int c = blockIdx.x, rows = forward_rows(a.T), E = a.E;
  const int lo = c * rows, hi = min(a.T, lo + rows);
  // the chunk's first rows and its picks are on their way before the sequences are known
  Row<kNI> next;
  int have = lo + group;
  if (a.logits && have < hi) load_row<kNI>(a.logits, have, E, j, next);
  int id[8];  // picks tid, tid + 256, ... of the chunk's at most 2048
  const int picks = (hi - lo) * a.topk;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    id[i] = tid + 256 * i < picks ? a.ids[static_cast<size_t>(lo) * a.topk + tid + 256 * i] : -1;
  const Starts seq(a.starts, a.n_seq, a.T);
  for (int b = seq.find(lo); b < a.n_seq; ++b) {
    const int s0 = max(lo, seq.at(b)), s1 = min(hi, seq.at(b + 1));
    if (s0 >= hi) break;
    if (s1 <= s0) continue;
    __syncthreads();
    cnt[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = tid + 256 * i;
      if (at >= (s0 - lo) * a.topk && at < (s1 - lo) * a.topk && id[i] >= 0 && id[i] < E)
        atomicAdd(&cnt[id[i]], 1);
    }
    if (a.logits) {
      float acc[4 * kNI] = {};
      int row = lo + (s0 - lo) / kPass * kPass + group;
      if (row != have && row < s1) load_row<kNI>(a.logits, row, E, j, next);
      for (; row < s1; row += kPass) {
        const Row<kNI> l = next;
        if (row + kPass < s1) load_row<kNI>(a.logits, row + kPass, E, j, next);
        Row<kNI> p, unused;
        row_scores<kNI, false>(l, a.score, p, unused);
        if (row >= s0) {
#pragma unroll
          for (int i = 0; i < 4 * kNI; ++i) acc[i] += p.v[i];
        }
      }
      have = -1;
#pragma unroll
      for (int i = 0; i < kNI; ++i)
        *reinterpret_cast<f32x4_t*>(&sums[group][64 * i + 4 * j]) =
            f32x4_t{acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]};
    }
    __syncthreads();
    if (tid < E) {
      const size_t at = static_cast<size_t>(c + b) * E + tid;
      float t[kPass];
      if (a.logits) {
#pragma unroll
        for (int i = 0; i < kPass; ++i) t[i] = sums[i][tid];
#pragma unroll
        for (int w = kPass / 2; w >= 1; w >>= 1)
#pragma unroll
          for (int i = 0; i < w; ++i) t[i] += t[i + w];
      }
      if constexpr (kOne) {
        store_through(&a.slot_counts[at], cnt[tid]);
        if (a.logits) store_through(&a.slot_probs[at], t[0]);
      } else {
        a.slot_counts[at] = cnt[tid];
        if (a.logits) a.slot_probs[at] = t[0];
      }
    }
  }
  if constexpr (kOne) {
    if (!last_workgroup(a.done)) return;
    // thread = expert; all slots at once (those no chunk met are not added)
    int n[kOneSlots];
    float p[kOneSlots];
    const int slots = static_cast<int>(gridDim.x) + a.n_seq;
#pragma unroll
    for (int i = 0; i < kOneSlots; ++i) {
      n[i] = 0;
      p[i] = 0.0f;
      if (i < slots && tid < E) {
        n[i] = load_through(&a.slot_counts[i * E + tid]);
        if (a.logits) p[i] = load_through(&a.slot_probs[i * E + tid]);
      }
    }
    double sum = 0.0;
    for (int b = 0; b < a.n_seq; ++b) {
      const int s0 = seq.at(b), s1 = seq.at(b + 1);
      const int first = s0 / rows + b, last = s1 > s0 ? (s1 - 1) / rows + b : -1;
      int count = 0;
      double prob = 0.0;
#pragma unroll
      for (int i = 0; i < kOneSlots; ++i) {
        if (i >= first && i <= last) {
          count += n[i];
          prob += p[i];
        }
      }
      const double len = s1 > s0 ? s1 - s0 : 1;
      prob /= len;
      if (tid < E) {
        a.counts[static_cast<size_t>(b) * E + tid] = count;
        if (a.loss) a.probs[static_cast<size_t>(b) * E + tid] = static_cast<float>(prob);
        sum += static_cast<double>(E) / (a.topk * len) * count * prob;
      }
    }
    if (!a.loss) return;
    __shared__ double part[4];
    sum = wave_sum_f64(sum);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    sum = (part[0] + part[1]) + (part[2] + part[3]);
    if (tid == 0) store_loss(a, sum);
  }
}

// a workgroup: every gridDim.x-th (b, kJ experts); the last one to finish adds the terms of the loss
template <int kJ>
__global__ __launch_bounds__(kReduce) void reduce_kernel(ForwardArgs a) {
  __shared__ double part[kReduce / kWave];
  const int groups = (a.E + kJ - 1) / kJ, items = a.n_seq * groups;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const double term = reduce_group<kJ>(a, i / groups, i % groups * kJ);
    if (a.loss && threadIdx.x == 0) store_through(&a.terms[i], term);
  }
  if (!a.loss) return;
  if (!last_workgroup(a.done)) return;
  double sum = 0.0;
  for (int i = threadIdx.x; i < items; i += kReduce) sum += load_through(&a.terms[i]);
  sum = wave_sum_f64(sum);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kReduce / kWave; ++i) sum += part[i];  // thread 0 holds part[0]
  store_loss(a, sum);
}

// ---------------------------------------------------------------- backward

template <int kNI>
__global__ __launch_bounds__(256) void backward_kernel(const float* __restrict__ logits,
                                                       const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ starts,
                                                       const float* __restrict__ dloss,
                                                       float* __restrict__ dlogits, int T, int E,
                                                       int topk, int n_seq, float coef,
                                                       int score) {
  const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int rows = backward_rows(T);
  const int lo = blockIdx.x * rows, hi = min(T, lo + rows);
  Row<kNI> next;
  int have = lo + group;
  if (have < hi) load_row<kNI>(logits, have, E, j, next);
  const float g = dloss ? *dloss : 1.0f;
  const Starts seq(starts, n_seq, T);
  for (int b = seq.find(lo); b < n_seq; ++b) {
    const int q0 = seq.at(b), q1 = seq.at(b + 1);
    const int s0 = max(lo, q0), s1 = min(hi, q1);
    if (s0 >= hi) break;
    if (s1 <= s0) continue;
    int row = lo + (s0 - lo) / kPass * kPass + group;
    if (row != have && row < s1) load_row<kNI>(logits, row, E, j, next);
    have = -1;
    const double len = q1 - q0;
    const float f =
        static_cast<float>(static_cast<double>(g) * coef / n_seq * E / (topk * len * len));
    // The gradient does not change with a constant taken off every count (the p of a
    // row add up to 1), so the counts are taken against the mean: near balance
    // a_j - sum a p would otherwise be a small difference of large terms.
    const int mean_count = static_cast<int>((2ll * topk * (q1 - q0) + E) / (2 * E));
    float a[4 * kNI];
#pragma unroll
    for (int i = 0; i < 4 * kNI; ++i) {
      const int e = 64 * (i >> 2) + 4 * j + (i & 3);
      a[i] = e < E ? f * static_cast<float>(counts[static_cast<size_t>(b) * E + e] - mean_count) : 0.0f;
    }
    for (; row < s1; row += kPass) {
      const Row<kNI> l = next;
      if (row + kPass < s1) load_row<kNI>(logits, row + kPass, E, j, next);
      Row<kNI> p, slope;
      row_scores<kNI, true>(l, score, p, slope);
      float mean = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * kNI; ++i) mean = __builtin_fmaf(a[i], p.v[i], mean);
      mean = row_sum(mean);
      if (row < s0) continue;  // the sequence in front's
      float* out = dlogits + static_cast<size_t>(row) * E;
#pragma unroll
      for (int i = 0; i < kNI; ++i) {
        const int e = 64 * i + 4 * j;
        f32x4_t v;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = slope.v[4 * i + c] * (a[4 * i + c] - mean);
        if (e + 4 <= E) {
          *reinterpret_cast<f32x4_any_t*>(out + e) = v;
        } else {
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (e + c < E) out[e + c] = v[c];
        }
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

// Most workgroups of the second launch: their counting is one after another. 256 /
// 512 / 2048 / one a group, with 16 experts: 256 sequences 95 / 87 / 96 / 116 us, 4000
// sequences 509 / 364 / 361 / 847.
constexpr int kReduceGroups = 512;

inline int chunks(const moe_balance_dims& d) {
  return (d.T + forward_rows(d.T) - 1) / forward_rows(d.T);
}
// 16 experts a workgroup of the second launch while that gives no more of them than
// CUs, else 64 (a slot line read whole, a quarter of the groups). Measured, us a
// forward and backward, 16 / 64: T = 65536, E = 256, 16 sequences 58.8 / 61.1, 32
// 63.3 / 61.2, 256 86 / 75; T = 20000, 4000 sequences 365 / 164.
inline int reduce_experts(const moe_balance_dims& d) {
  return d.n_seq * ((d.E + 15) / 16) <= 256 ? 16 : 64;
}
inline int reduce_items(const moe_balance_dims& d) {
  return d.n_seq * ((d.E + reduce_experts(d) - 1) / reduce_experts(d));
}

// workspace: the done counter (zero between calls), the loss terms, the slots
struct BalanceLayout {
  size_t terms, counts, probs, total;
};

BalanceLayout balance_layout(const moe_balance_dims& d) {
  BalanceLayout l;
  const size_t slots = static_cast<size_t>(chunks(d) + d.n_seq) * d.E;
  l.terms = 256;
  l.counts = l.terms + round_up(static_cast<size_t>(reduce_items(d)) * 8, 256);
  l.probs = l.counts + round_up(slots * 4, 256);
  l.total = l.probs + round_up(slots * 4, 256);
  return l;
}

template <int kNI>
void launch_forward(const ForwardArgs& a, const moe_balance_dims& m, hipStream_t stream) {
  const int n_chunks = chunks(m);
  if (n_chunks + a.n_seq <= kOneSlots) {
    chunk_kernel<kNI, true><<<n_chunks, 256, 0, stream>>>(a);
    return;
  }
  chunk_kernel<kNI, false><<<n_chunks, 256, 0, stream>>>(a);
  const int items = reduce_items(m), grid = items < kReduceGroups ? items : kReduceGroups;
  if (reduce_experts(m) == 64)
    reduce_kernel<64><<<grid, kReduce, 0, stream>>>(a);
  else
    reduce_kernel<16><<<grid, kReduce, 0, stream>>>(a);
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
  ForwardArgs a;
  a.logits = logits, a.ids = topk_ids, a.starts = seq_starts;
  a.slot_counts = reinterpret_cast<int32_t*>(ws + l.counts);
  a.slot_probs = reinterpret_cast<float*>(ws + l.probs);
  a.counts = counts, a.probs = probs, a.loss = loss;
  a.terms = reinterpret_cast<double*>(ws + l.terms), a.done = reinterpret_cast<int32_t*>(ws);
  a.T = m.T, a.E = m.E, a.topk = m.topk, a.n_seq = m.n_seq, a.score = m.score, a.coef = m.coef;
  if (m.E <= 64)
    launch_forward<1>(a, m, stream);
  else if (m.E <= 128)
    launch_forward<2>(a, m, stream);
  else
    launch_forward<4>(a, m, stream);
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
  const moe_balance_dims& m = *dims;
  const unsigned grid = (m.T + backward_rows(m.T) - 1) / backward_rows(m.T);
  const auto launch = [&](auto kernel) {
    kernel<<<grid, 256, 0, stream>>>(logits, counts, seq_starts, dloss, dlogits, m.T, m.E, m.topk,
                                     m.n_seq, m.coef, m.score);
  };
  if (m.E <= 64)
    launch(backward_kernel<1>);
  else if (m.E <= 128)
    launch(backward_kernel<2>);
  else
    launch(backward_kernel<4>);
  return launch_status();
}

}  // extern "C"
