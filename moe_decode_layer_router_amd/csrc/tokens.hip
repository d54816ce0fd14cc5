// tokens.hip -- the picks of many rows sorted by local expert (moe_sort), the
// tokens' rows brought into that order (moe_dispatch) and back as weighted sums
// (moe_return), and the gradient (moe_return_backward).
#include <type_traits>

#include "common.h"
#include "host.h"

namespace moeblk {
namespace {

// ---------------------------------------------------------------- sort
//
// A stable counting sort of the picks by local expert. Workgroups take chunks of
// picks, a chunk's waves consecutive runs of 64. With several chunks a launch in
// front counts each chunk's picks per expert; every workgroup then adds up the
// chunks in front of its own. Within a run, a pick's rank among those of its
// expert is a match over the bits of the expert's index (one ballot a bit). All
// counts are integers, so no order of atomics shows. Latency bounds it: 512 picks 3.9 us in
// one launch, 65536 picks 4.7 + 5.4 us, 524288 picks 11.7 us in all (256 experts held 13.8), 2^25 picks
// 258 (762; 79 by the bytes): a wave then makes up to 128 rounds, one load of ids in flight.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kMaxLocal = 256, kMaxChunks = 256;
constexpr int kMinChunk = 2 * kSortThreads;  // picks

__host__ __device__ inline int sort_chunk(int picks) {
  const int per = (picks + kMaxChunks - 1) / kMaxChunks;
  const int c = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
  return c < kMinChunk ? kMinChunk : c;
}
inline int sort_chunks(int picks) { return (picks + sort_chunk(picks) - 1) / sort_chunk(picks); }

struct SortArgs {
  const int32_t* ids;
  int32_t *counts, *offsets, *rows, *pick_pos;
  int32_t* hist;  // [chunks][n]
  int picks, topk, n, base, chunk, chunks;
};

// the local expert of a pick, or -1
__device__ __forceinline__ int local_of(const SortArgs& a, int p, int end) {
  if (p >= end) return -1;
  const int e = a.ids[p] - a.base;
  return e >= 0 && e < a.n ? e : -1;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int cnt[kMaxLocal];
  const int tid = threadIdx.x, c = blockIdx.x;
  const int64_t lo = static_cast<int64_t>(c) * a.chunk;
  const int end = static_cast<int>(lo + a.chunk < a.picks ? lo + a.chunk : a.picks);
  if (tid < kMaxLocal) cnt[tid] = 0;
  __syncthreads();
  for (int p = static_cast<int>(lo) + tid; p < end; p += kSortThreads) {
    const int e = local_of(a, p, end);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < a.n) a.hist[c * a.n + tid] = cnt[tid];
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ int at[kSortWaves][kMaxLocal];  // counts of a wave's run, then its next positions
  __shared__ int before[4][kMaxLocal], all[4][kMaxLocal];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = blockIdx.x, n = a.n;
  const int lo = c * a.chunk, end = min(lo + a.chunk, a.picks);
  const int run = a.chunk / kSortWaves;  // a multiple of 64
  const int w0 = lo + wave * run, w1 = min(w0 + run, end);
  for (int i = tid; i < kSortWaves * kMaxLocal; i += kSortThreads) (&at[0][0])[i] = 0;
  __syncthreads();
  for (int p = w0 + lane; p < w1; p += kWave) {
    const int e = local_of(a, p, w1);
    if (e >= 0) atomicAdd(&at[wave][e], 1);
  }
  // picks of the chunks in front of this one, and of all: expert tid % 256, a quarter
  // of the chunks each
  {
    const int e = tid & (kMaxLocal - 1), q = tid / kMaxLocal;
    int b = 0, s = 0;
    if (e < n && a.chunks > 1) {
#pragma unroll 8
      for (int i = q; i < a.chunks; i += 4) {
        const int v = a.hist[i * n + e];
        s += v;
        if (i < c) b += v;
      }
    }
    before[q][e] = b;
    all[q][e] = s;
  }
  __syncthreads();
  __shared__ int start[kMaxLocal + 1], wave_total[4];
  int mine = 0, incl = 0;
  if (tid < kMaxLocal) {
    if (a.chunks > 1) {
      mine = all[0][tid] + all[1][tid] + all[2][tid] + all[3][tid];
    } else {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) mine += at[w][tid];
    }
    incl = mine;  // inclusive prefix sum over the experts
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) {
      const int v = __shfl_up(incl, s, kWave);
      if (lane >= s) incl += v;
    }
    if (lane == 63) wave_total[wave] = incl;
  }
  __syncthreads();
  if (tid < kMaxLocal) {
    for (int w = 0; w < wave; ++w) incl += wave_total[w];
    start[tid + 1] = incl;
    if (tid == 0) start[0] = 0;
    if (c == 0 && tid < n) {
      a.counts[tid] = mine;
      a.offsets[tid + 1] = incl;
      if (tid == 0) a.offsets[0] = 0;
    }
    // the first position of each wave's run
    int p = incl - mine + before[0][tid] + before[1][tid] + before[2][tid] + before[3][tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int k = at[w][tid];
      at[w][tid] = p;
      p += k;
    }
  }
  __syncthreads();
  const int total = start[n];
  int bits = 0;
  while ((1 << bits) < n) ++bits;
  const uint64_t below = (1ull << lane) - 1;
  for (int p0 = w0; p0 < w1; p0 += kWave) {
    const int p = p0 + lane, e = local_of(a, p, w1);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool set = (e >> b) & 1;
      const uint64_t m = __ballot(set);
      same &= set ? m : ~m;
    }
    int pos = -1;
    if (e >= 0) pos = at[wave][e] + __builtin_popcountll(same & below);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && (same & below) == 0) at[wave][e] += __builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (p < w1) {
      a.pick_pos[p] = pos;
      if (pos >= 0) a.rows[pos] = p / a.topk;
    }
  }
  // positions that no pick has
  for (int p = max(lo, total) + tid; p < end; p += kSortThreads) a.rows[p] = -1;
}

// ---------------------------------------------------------------- rows
//
// Rows move in pieces of 16 bytes of the wider type, 8 bf16 values or 4: kLanes threads
// take a token's row, every kLanes-th piece each, so that a wave's accesses are contiguous and
// a token's row is read once for all of its picks. Rows of any length start anywhere:
// accesses take any alignment. All of it is bound by memory: 8192 x 7168, fp32 tokens, bf16
// rows, 32 of 256 experts held, dispatch and return one behind the other 57 and 72 us (352 MB
// each, 6.2 and 4.9 TB/s); 4096 x 4096 bf16, all 8 picks held, the gradient 113 us (570 MB, 5.0
// TB/s), the return without weights 57 (302 MB, 5.3 TB/s).
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any4_t __attribute__((aligned(4)));

template <int kN>
struct Piece {
  float v[kN];
};
template <typename Tok, typename Row>
constexpr int kPiece = sizeof(Tok) + sizeof(Row) == 4 ? 8 : 4;

// a piece as loaded; behind the row's end: zeros
template <typename T, int kN>
struct Raw {
  uint32_t w[kN * sizeof(T) / 4];
};

template <typename T, int kN>
__device__ __forceinline__ Raw<T, kN> load_raw(const T* row, int c, int d) {
  Raw<T, kN> r;
  if (c + kN <= d) {
    if constexpr (kN * sizeof(T) >= 16) {
#pragma unroll
      for (int h = 0; h < static_cast<int>(kN * sizeof(T) / 16); ++h) {
        const u32x4_t u = *reinterpret_cast<const u32x4_any_t*>(row + c + 16 / sizeof(T) * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[4 * h + i] = u[i];
      }
    } else {
      static_assert(kN * sizeof(T) == 8, "8, 16 or 32 bytes");
      const u32x2_t u = *reinterpret_cast<const u32x2_any_t*>(row + c);
      r.w[0] = u[0];
      r.w[1] = u[1];
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < static_cast<int>(kN * sizeof(T) / 4); ++i) r.w[i] = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (c + i >= d) continue;
    if constexpr (sizeof(T) == 2)
      r.w[i >> 1] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
    else
      r.w[i] = __float_as_uint(row[c + i]);
  }
  return r;
}
template <typename T, int kN>
__device__ __forceinline__ Piece<kN> values(const Raw<T, kN>& r) {
  Piece<kN> p;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if constexpr (sizeof(T) == 2)
      p.v[i] = i & 1 ? bf16_hi(r.w[i >> 1]) : bf16_lo(r.w[i >> 1]);
    else
      p.v[i] = __uint_as_float(r.w[i]);
  }
  return p;
}

// Stores go past the caches: 8192 x 7168, bf16 rows, fp32 tokens, 32 of 256 experts held, us with
// / without: moe_return 54 / 82, moe_dispatch 51 / 58.
template <int kN>
__device__ __forceinline__ void store_piece(uint16_t* row, int c, int d, const Piece<kN>& p) {
  uint32_t q[kN / 2];
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) q[i] = pack_bf16x2(p.v[2 * i], p.v[2 * i + 1]);
  if (c + kN <= d) {
    if constexpr (kN == 8)
      __builtin_nontemporal_store(u32x4_t{q[0], q[1], q[2], q[3]}, reinterpret_cast<u32x4_any_t*>(row + c));
    else
      __builtin_nontemporal_store(u32x2_t{q[0], q[1]}, reinterpret_cast<u32x2_any_t*>(row + c));
  } else {
#pragma unroll
    for (int i = 0; i < kN - 1; ++i)
      if (c + i < d) row[c + i] = static_cast<uint16_t>(q[i >> 1] >> (16 * (i & 1)));
  }
}
template <int kN>
__device__ __forceinline__ void store_piece(float* row, int c, int d, const Piece<kN>& p) {
  if (c + kN <= d) {
    __builtin_nontemporal_store(f32x4_t{p.v[0], p.v[1], p.v[2], p.v[3]}, reinterpret_cast<f32x4_any4_t*>(row + c));
  } else {
#pragma unroll
    for (int i = 0; i < kN - 1; ++i)
      if (c + i < d) row[c + i] = p.v[i];
  }
}

struct RowsArgs {
  const int32_t* pick_pos;
  const float* w;       // NULL: ones
  const void *tok, *row;  // inputs of either side
  void *tok_out, *row_out;
  float* dw;
  int T, topk, d, R;
};

// The positions of a token's picks; a position outside the sorted rows is none. With a wave
// or more a row they are the same in the whole wave, and known to be.
template <int kLanes>
__device__ __forceinline__ void load_pos(const RowsArgs& a, int t, int (&pos)[8]) {
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    pos[s] = s < a.topk ? a.pick_pos[static_cast<size_t>(t) * a.topk + s] : -1;
    if (pos[s] >= a.R) pos[s] = -1;
    if constexpr (kLanes >= kWave) pos[s] = __builtin_amdgcn_readfirstlane(pos[s]);
  }
}

template <typename Tok, typename Row, int kLanes>
__global__ __launch_bounds__(256) void dispatch_kernel(RowsArgs a) {
  constexpr int kN = kPiece<Tok, Row>;
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  if (t >= a.T) return;
  int pos[8];
  load_pos<kLanes>(a, t, pos);
  bool any = false;  // rows of tokens without a pick are not read
#pragma unroll
  for (int s = 0; s < 8; ++s) any = any || pos[s] >= 0;
  if (!any) return;
  const Tok* x = static_cast<const Tok*>(a.tok) + static_cast<size_t>(t) * a.d;
  for (int c = threadIdx.x % kLanes * kN; c < a.d; c += kLanes * kN) {
    const Piece<kN> p = values<Tok, kN>(load_raw<Tok, kN>(x, c, a.d));
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (pos[s] >= 0)
        store_piece(static_cast<Row*>(a.row_out) + static_cast<size_t>(pos[s]) * a.d, c, a.d, p);
  }
}

// the pieces of all picks' rows, their loads in flight together
template <typename Row, int kN>
__device__ __forceinline__ void load_rows(const RowsArgs& a, const int (&pos)[8], int c, Raw<Row, kN> (&y)[8]) {
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (pos[s] >= 0)
      y[s] = load_raw<Row, kN>(static_cast<const Row*>(a.row) + static_cast<size_t>(pos[s]) * a.d, c, a.d);
}

// sums in fp32, in slot order, one rounding
template <typename Tok, typename Row, int kLanes>
__global__ __launch_bounds__(256) void return_kernel(RowsArgs a) {
  constexpr int kN = kPiece<Tok, Row>;
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  if (t >= a.T) return;
  int pos[8];
  float w[8];
  load_pos<kLanes>(a, t, pos);
#pragma unroll
  for (int s = 0; s < 8; ++s)
    w[s] = a.w && pos[s] >= 0 ? a.w[static_cast<size_t>(t) * a.topk + s] : 1.0f;
  Tok* out = static_cast<Tok*>(a.tok_out) + static_cast<size_t>(t) * a.d;
  for (int c = threadIdx.x % kLanes * kN; c < a.d; c += kLanes * kN) {
    Raw<Row, kN> y[8];
    load_rows(a, pos, c, y);
    Piece<kN> sum = {};
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (pos[s] < 0) continue;
      const Piece<kN> p = values<Row, kN>(y[s]);
#pragma unroll
      for (int i = 0; i < kN; ++i) sum.v[i] = __builtin_fmaf(p.v[i], w[s], sum.v[i]);
    }
    store_piece(out, c, a.d, sum);
  }
}

// dy = w dout, dw = <dout, y>: the row of dout is read once for all picks; the
// threads' fp32 sums are added in a fixed tree
template <typename Tok, typename Row, int kLanes>
__global__ __launch_bounds__(256) void return_backward_kernel(RowsArgs a) {
  constexpr int kN = 16 / sizeof(Row);  // the rows' bytes, read and written, are most of all
  __shared__ float red[256 / kWave][8];
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const bool in = t < a.T;
  int pos[8];
  float w[8], dw[8];
  load_pos<kLanes>(a, in ? t : 0, pos);
  bool any = false;  // rows of tokens without a pick are not read
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    if (!in) pos[s] = -1;
    any = any || pos[s] >= 0;
    w[s] = pos[s] >= 0 ? a.w[static_cast<size_t>(t) * a.topk + s] : 1.0f;
    dw[s] = 0.0f;
  }
  const Tok* g = static_cast<const Tok*>(a.tok) + static_cast<size_t>(in ? t : 0) * a.d;
  for (int c = threadIdx.x % kLanes * kN; any && c < a.d; c += kLanes * kN) {
    const Raw<Tok, kN> graw = load_raw<Tok, kN>(g, c, a.d);
    Raw<Row, kN> y[8];
    load_rows(a, pos, c, y);
    const Piece<kN> p = values<Tok, kN>(graw);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (pos[s] < 0) continue;
      const Piece<kN> v = values<Row, kN>(y[s]);
      Piece<kN> q;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        dw[s] = __builtin_fmaf(p.v[i], v.v[i], dw[s]);
        q.v[i] = p.v[i] * w[s];
      }
      store_piece(static_cast<Row*>(a.row_out) + static_cast<size_t>(pos[s]) * a.d, c, a.d, q);
    }
  }
#pragma unroll
  for (int s = 0; s < 8; ++s)
#pragma unroll
    for (int m = (kLanes < kWave ? kLanes : kWave) / 2; m >= 1; m >>= 1)
      dw[s] += __shfl_xor(dw[s], m, kWave);
  if constexpr (kLanes > kWave) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int s = 0; s < 8; ++s) red[threadIdx.x >> 6][s] = dw[s];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      dw[s] = red[0][s];
#pragma unroll
      for (int v = 1; v < 256 / kWave; ++v) dw[s] += red[v][s];
    }
  }
  const int s = threadIdx.x % kLanes;
  float mine = dw[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mine = s == i ? dw[i] : mine;
  if (in && s < a.topk) a.dw[static_cast<size_t>(t) * a.topk + s] = mine;
}

// threads a row: 16, 64 or a workgroup's 256, about a piece each
template <typename F>
void for_lanes(int d, F f) {
  if (d <= 128)
    f(std::integral_constant<int, 16>());
  else if (d <= 1024)
    f(std::integral_constant<int, 64>());
  else
    f(std::integral_constant<int, 256>());
}
template <typename F>
void for_types(const moe_rows_dims& m, F f) {
  const auto row = [&](auto tok) {
    if (m.row_type == MOE_BF16) f(tok, uint16_t());
    else f(tok, float());
  };
  if (m.tok_type == MOE_BF16) row(uint16_t());
  else row(float());
}
template <int kLanes>
unsigned rows_grid(int T) {
  return static_cast<unsigned>((static_cast<int64_t>(T) * kLanes + 255) / 256);
}

size_t sort_workspace(const moe_rows_dims& m) {
  const int chunks = sort_chunks(m.T * m.topk);
  return round_up(static_cast<size_t>(chunks) * m.n_local * 4, 256);
}

}  // namespace

int check_rows_dims(const moe_rows_dims* d) {
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL);
  MOE_REQUIRE(d->T >= 1 && d->T <= 1 << 22, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->E >= 1 && d->E <= kMaxLocal, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->topk >= 1 && d->topk <= 8 && d->topk <= d->E, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->n_local >= 1 && d->local_base >= 0 && d->local_base <= d->E &&
                  d->n_local <= d->E - d->local_base,
              MOE_ERR_SHAPE);
  MOE_REQUIRE(d->d >= 1 && d->d <= 16384, MOE_ERR_SHAPE);
  MOE_REQUIRE(d->tok_type == MOE_BF16 || d->tok_type == MOE_FP32, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(d->row_type == MOE_BF16 || d->row_type == MOE_FP32, MOE_ERR_UNSUPPORTED);
  return MOE_OK;
}

}  // namespace moeblk

using namespace moeblk;

extern "C" {

int moe_check_rows_dims(const moe_rows_dims* dims) { return check_rows_dims(dims); }

size_t moe_sort_workspace_bytes(const moe_rows_dims* dims) {
  return check_rows_dims(dims) ? 0 : sort_workspace(*dims);
}

int moe_sort(const moe_rows_dims* dims, const int32_t* topk_ids, int32_t* counts, int32_t* offsets,
             int32_t* rows, int32_t* pick_pos, void* workspace, size_t workspace_bytes,
             hipStream_t stream) {
  const int rc = check_rows_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(topk_ids && counts && offsets && rows && pick_pos && workspace, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(topk_ids) && aligned16(counts) && aligned16(offsets) && aligned16(rows) &&
                  aligned16(pick_pos) && aligned16(workspace),
              MOE_ERR_ALIGN);
  MOE_REQUIRE(workspace_bytes >= sort_workspace(*dims), MOE_ERR_WORKSPACE);
  const int picks = dims->T * dims->topk;
  const SortArgs a = {topk_ids,      counts,        offsets,          rows,
                      pick_pos,      static_cast<int32_t*>(workspace), picks,
                      dims->topk,    dims->n_local, dims->local_base, sort_chunk(picks),
                      sort_chunks(picks)};
  if (a.chunks > 1) sort_count_kernel<<<a.chunks, kSortThreads, 0, stream>>>(a);
  sort_place_kernel<<<a.chunks, kSortThreads, 0, stream>>>(a);
  return launch_status();
}

int moe_dispatch(const moe_rows_dims* dims, const void* x, const int32_t* pick_pos, void* xs,
                 hipStream_t stream) {
  const int rc = check_rows_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(x && pick_pos && xs, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(x) && aligned16(pick_pos) && aligned16(xs), MOE_ERR_ALIGN);
  const RowsArgs a = {pick_pos, nullptr, x,       nullptr,    nullptr, xs,
                      nullptr,  dims->T, dims->topk, dims->d, dims->T * dims->topk};
  for_types(*dims, [&](auto tok, auto row) {
    for_lanes(dims->d, [&](auto n) {
      constexpr int kLanes = decltype(n)::value;
      dispatch_kernel<decltype(tok), decltype(row), kLanes>
          <<<rows_grid<kLanes>(dims->T), 256, 0, stream>>>(a);
    });
  });
  return launch_status();
}

int moe_return(const moe_rows_dims* dims, const void* y, const float* topk_w,
               const int32_t* pick_pos, void* out, hipStream_t stream) {
  const int rc = check_rows_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(y && pick_pos && out, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(y) && aligned16(topk_w) && aligned16(pick_pos) && aligned16(out),
              MOE_ERR_ALIGN);
  const RowsArgs a = {pick_pos, topk_w,  nullptr,    y,       out, nullptr,
                      nullptr,  dims->T, dims->topk, dims->d, dims->T * dims->topk};
  for_types(*dims, [&](auto tok, auto row) {
    for_lanes(dims->d, [&](auto n) {
      constexpr int kLanes = decltype(n)::value;
      return_kernel<decltype(tok), decltype(row), kLanes>
          <<<rows_grid<kLanes>(dims->T), 256, 0, stream>>>(a);
    });
  });
  return launch_status();
}

int moe_return_backward(const moe_rows_dims* dims, const void* dout, const void* y,
                        const float* topk_w, const int32_t* pick_pos, void* dy, float* dtopk_w,
                        hipStream_t stream) {
  const int rc = check_rows_dims(dims);
  if (rc) return rc;
  MOE_REQUIRE(dout && y && topk_w && pick_pos && dy && dtopk_w, MOE_ERR_NULL);
  MOE_REQUIRE(aligned16(dout) && aligned16(y) && aligned16(topk_w) && aligned16(pick_pos) &&
                  aligned16(dy) && aligned16(dtopk_w),
              MOE_ERR_ALIGN);
  const RowsArgs a = {pick_pos, topk_w,  dout,       y,       nullptr, dy,
                      dtopk_w,  dims->T, dims->topk, dims->d, dims->T * dims->topk};
  for_types(*dims, [&](auto tok, auto row) {
    for_lanes(dims->d, [&](auto n) {
      constexpr int kLanes = decltype(n)::value;
      return_backward_kernel<decltype(tok), decltype(row), kLanes>
          <<<rows_grid<kLanes>(dims->T), 256, 0, stream>>>(a);
    });
  });
  return launch_status();
}

}  // extern "C"
