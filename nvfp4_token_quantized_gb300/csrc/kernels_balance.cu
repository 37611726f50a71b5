// kernels_balance.cu - the balance loss of the expert choice, the counts of
// the chosen experts, and the loss's gradient.
//
// A token's shares p are its softmax, or its sigmoid scores over their sum.
// The loss of a sequence of N tokens is coefficient * E / (K N^2) times the sum
// over the experts of (times chosen) * (sum of p), so one pass over the logits
// leaves E sums and E counts a run of rows, which a second, small kernel joins
// in the order of the runs: no atomics on floats, the same bits every time.  The
// roundings of tokens alike all go one way, so no FP32 chain grows with the batch: a
// lane adds 32 rows at a time, a run is one such sum (128 experts and fewer) or up to
// 32, a thread of the join keeps what each addition rounds away (add_kept), and the
// threads' sums meet in a tree.  (1048576 rows FP32, runs of one sum or of more: 64
// experts 87 and 103 us, 256 experts 188 and 167: few CTAs an SM gain by fewer starts,
// many lose by the longer code.)
//
// Sixteen lanes share a row: four experts a lane and chunk, so that a row of
// 256 takes four 16-byte loads a lane and two trees of four steps for a
// maximum and a sum, and the lanes' own sums over the rows stay in registers.
//
// Bound by the bytes of the logits.  131072 x 256 FP32: the sums 25 us (138 MB, 5.4
// TB/s with a launch's ramp and drain), their join 8, the gradient 38.5 (268 MB,
// 7 TB/s: part of what it writes stays in L2), 56 with rows to add to (403 MB, 7.3
// TB/s).  A few thousand rows in many sequences are a chain of latencies: 32768 x
// 160 bf16 in 41 sequences 33 us, loss and gradient.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "elem_types.cuh"
#include "kernels_ops.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int ROWS_AT_ONCE = 2 * WARPS;  // sixteen lanes a row
constexpr int SUM_ROWS = 32 * ROWS_AT_ONCE;  // that a CTA adds before its lanes' sums are kept
constexpr int LONG_RUNS = 2;             // of more than so many 64 experts: several such sums
constexpr int JOIN = 8;                  // CTAs of a cluster that joins the runs' sums
constexpr int JOIN_THREADS = 1024;       // of a CTA that joins all runs of a batch
constexpr int OFFSETS = 1024;            // that a CTA keeps in shared memory
constexpr unsigned ALL = 0xffffffffu;

// Four neighbouring elements of a row, as loaded.
template <typename T>
using Quad = std::conditional_t<sizeof(T) == 4, uint4, uint2>;

template <typename T>
__device__ __forceinline__ uint32_t minus_infinity();
template <>
__device__ __forceinline__ uint32_t minus_infinity<float>() {
  return 0xff800000u;
}
template <>
__device__ __forceinline__ uint32_t minus_infinity<__half>() {
  return 0xfc00fc00u;
}
template <>
__device__ __forceinline__ uint32_t minus_infinity<__nv_bfloat16>() {
  return 0xff80ff80u;
}
template <typename T>
__device__ __forceinline__ void fill(uint4& q, uint32_t v) {
  q = make_uint4(v, v, v, v);
}
template <typename T>
__device__ __forceinline__ void fill(uint2& q, uint32_t v) {
  q = make_uint2(v, v);
}
template <typename T>
__device__ __forceinline__ void widen(const uint4& q, float* x) {
  x[0] = __uint_as_float(q.x), x[1] = __uint_as_float(q.y), x[2] = __uint_as_float(q.z), x[3] = __uint_as_float(q.w);
}
template <typename T>
__device__ __forceinline__ void widen(const uint2& q, float* x) {
  const float2 a = unpack2(q.x, T()), b = unpack2(q.y, T());
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
template <typename T>
__device__ __forceinline__ Quad<T> narrow(const float* x) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  else
    return make_uint2(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()));
}

// A lane's elements of one row as they were loaded (what the lane has no
// expert for, or no row, reads `other`).  VEC: rows of four-element loads;
// otherwise the lanes take neighbouring elements.
template <typename T, bool VEC, int C>
struct RowPart {
  static constexpr int N = 4 * C;
  Quad<T> q[VEC ? C : 1];
  T v[VEC ? 1 : N];
  __device__ __forceinline__ static int expert(int i, int sub) { return VEC ? (i >> 2) * 64 + sub * 4 + (i & 3) : i * 16 + sub; }
  // other: the bits that stand for a missing element (two of a 16-bit type)
  __device__ __forceinline__ void load(const T* row, int E, int sub, bool on, uint32_t other) {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = c * 64 + sub * 4;
        fill<T>(q[c], other);
        if (on && e < E) q[c] = *reinterpret_cast<const Quad<T>*>(row + e);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = i * 16 + sub;
        v[i] = from_f32<T>(other ? -INFINITY : 0.0f);
        if (on && e < E) v[i] = row[e];
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[N]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < C; ++c) widen<T>(q[c], x + 4 * c);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = to_f32(v[i]);
    }
  }
  __device__ __forceinline__ static void store(T* row, int E, int sub, const float (&x)[N]) {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = c * 64 + sub * 4;
        if (e < E) *reinterpret_cast<Quad<T>*>(row + e) = narrow<T>(x + 4 * c);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * 16 + sub < E) row[i * 16 + sub] = from_f32<T>(x[i]);
    }
  }
};

// Over the sixteen lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
  return v;
}

// The hardware's exponential and reciprocal, results below 2^-126 as 0: without
// that they take twice the instructions, which bound large batches beside the
// bytes.
__device__ __forceinline__ float exponential(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.44269504f));
  return r;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// x becomes scores that are the shares times their sum; returns 1 / sum, 0
// for a row of closed experts.  (Some 2^-22 of a score; the logits' distance from
// the maximum times 2^-24 more.)
template <int N>
__device__ __forceinline__ float softmax_scores(float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
  m = row_max(m);
  if (m == -INFINITY) m = 0.0f;
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = exponential(x[i] - m);
    total += x[i];
  }
  total = row_sum(total);
  return total == 0.0f ? 0.0f : reciprocal(total);
}
// The same for sigmoid scores, with the sum's own 1e-20; rest, if wanted, gets
// 1 - s, without the cancellation.
template <int N, bool REST>
__device__ __forceinline__ float sigmoid_scores(float (&x)[N], float (&rest)[REST ? N : 1]) {
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = exponential(-fabsf(x[i]));
    const float r = reciprocal(1.0f + a);
    const bool up = x[i] >= 0.0f;
    if constexpr (REST) rest[i] = up ? a * r : r;
    x[i] = up ? r : a * r;
    total += x[i];
  }
  return reciprocal(row_sum(total) + SELECT_SUM_EPS);
}

// ---- runs of rows ----

// Rows [lo, hi) of one sequence, or (seq < 0) of none.
struct Run {
  int64_t lo, hi, seq;
};

__device__ __forceinline__ int64_t bound_of(const BalanceArgs& a, int64_t i) {
  const int64_t v = a.offsets[i];
  return v < 0 ? 0 : v > a.rows ? a.rows : v;
}

// A CTA's walk through the sequences; the first offsets are kept in shared
// memory, which spares every step one latency of L2.
struct Walk {
  int bounds[OFFSETS];
  int count;
  // The sequence that row `row` lies in or before: the number of ends at or
  // before it, counted by all threads.
  __device__ __forceinline__ int64_t first(const BalanceArgs& a, int64_t row) {
    if (!a.offsets) return 0;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    int n = 0;
    for (int64_t i = threadIdx.x; i <= a.sequences; i += THREADS) {
      const int64_t v = bound_of(a, i);
      if (i < OFFSETS) bounds[i] = (int)v;
      n += i > 0 && v <= row;
    }
    n = __reduce_add_sync(ALL, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&count, n);
    __syncthreads();
    return count;
  }
  __device__ __forceinline__ int64_t at(const BalanceArgs& a, int64_t i) const {
    return i < OFFSETS ? bounds[i] : bound_of(a, i);
  }
  // The run that starts at row `from` < end; seq moves on to its sequence.  It
  // ends behind `from` whatever the offsets hold.
  __device__ __forceinline__ Run next(const BalanceArgs& a, int64_t from, int64_t end, int64_t& seq) const {
    if (!a.offsets) return {from, end, 0};
    while (seq < a.sequences && at(a, seq + 1) <= from) ++seq;
    if (seq >= a.sequences) return {from, end, -1};
    const int64_t lo = at(a, seq), hi = at(a, seq + 1);
    if (from < lo) return {from, lo < end ? lo : end, -1};
    return {from, hi < end ? hi : end, seq};
  }
};

// Words of a run's sums: E sums of shares, E counts, the tokens.
__host__ __device__ __forceinline__ int part_words(int E) { return 2 * E + 1; }

template <int THREADS>
struct JoinShared {
  float sums[THREADS];
  int counts[THREADS];
  int tokens;
  float loss;
};
struct SumShared {
  float sums[WARPS][SELECT_MAX_EXPERTS];
  int counts[SELECT_MAX_EXPERTS];
  int tokens;
};
struct SmallShared {  // of a cluster that joins its own sums
  uint32_t part[2 * SELECT_MAX_EXPERTS + 1];
  JoinShared<THREADS> join;
};

// Sums and counts of rows [lo, hi) into dst (global or shared).
template <typename T, bool VEC, int C>
__device__ __forceinline__ void sum_run(const BalanceArgs& a, int64_t lo, int64_t hi, SumShared& sh, uint32_t* dst) {
  using Part = RowPart<T, VEC, C>;
  constexpr int N = Part::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 15, half = lane >> 4;
  for (int e = threadIdx.x; e < a.E; e += THREADS) sh.counts[e] = 0;
  if (threadIdx.x == 0) sh.tokens = 0;
  __syncthreads();

  const T* logits = static_cast<const T*>(a.logits);
  // (a lane also brings slots sub and sub + 16 of its row's chosen experts)
  const auto fetch = [&](int64_t row, Part& p, int (&id)[2]) {
    const bool in = row < hi;
    const bool on = in && (!a.mask || a.mask[row]);  // (a load beside the others, not before them)
    p.load(logits + row * a.stride, a.E, sub, in, minus_infinity<T>());
    id[0] = in && sub < a.K ? a.ids[row * a.K + sub] : -1;
    id[1] = in && sub + 16 < a.K ? a.ids[row * a.K + sub + 16] : -1;
    return on;
  };
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  int mine = 0;
  Part cur;
  int id[2];
  bool on = fetch(lo + warp * 2 + half, cur, id);
  constexpr bool LONG = C > LONG_RUNS;
  int64_t base = lo + warp * 2;
  bool kept = false;
  do {
    for (const int64_t stop = LONG ? min(base + SUM_ROWS, hi) : hi; base < stop; base += ROWS_AT_ONCE) {
      Part nxt;
      int nxt_id[2];
      const bool nxt_on = fetch(base + ROWS_AT_ONCE + half, nxt, nxt_id);
      if (on && (unsigned)id[0] < (unsigned)a.E) atomicAdd(&sh.counts[id[0]], 1);
      if (on && (unsigned)id[1] < (unsigned)a.E) atomicAdd(&sh.counts[id[1]], 1);
      float x[N];
      cur.values(x);
      if (a.mask && !on) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = -INFINITY;
      }
      float none[1], inv;
      if (a.sigmoid)
        inv = sigmoid_scores<N, false>(x, none);
      else
        inv = softmax_scores(x);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
      mine += on;
      cur = nxt;
      on = nxt_on;
      id[0] = nxt_id[0];
      id[1] = nxt_id[1];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      acc[i] += __shfl_xor_sync(ALL, acc[i], 16);
      const int e = Part::expert(i, sub);
      if (half == 0 && e < a.E) sh.sums[warp][e] = kept ? sh.sums[warp][e] + acc[i] : acc[i];
      acc[i] = 0.0f;
    }
    kept = true;
  } while (LONG && base < hi);
  if (sub == 0 && mine) atomicAdd(&sh.tokens, mine);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sh.sums[w][e];
    dst[e] = __float_as_uint(s);
    dst[a.E + e] = (uint32_t)sh.counts[e];
  }
  if (threadIdx.x == 0) dst[2 * a.E] = (uint32_t)sh.tokens;
  __syncthreads();
}

// Joins `parts` runs' sums of sequence s: the cluster's CTAs take an eighth of
// the experts each, and in a CTA groups of threads every so many runs.
template <int THREADS, typename PartAt>
__device__ __forceinline__ void join_parts(const BalanceArgs& a, int64_t s, int parts, PartAt part_at,
                                           JoinShared<THREADS>& sh) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int width = (a.E + JOIN - 1) / JOIN, groups = THREADS / width;
  const int local = threadIdx.x % width, group = threadIdx.x / width, e = rank * width + local;
  if (threadIdx.x == 0) sh.tokens = 0;
  __syncthreads();
  float sum = 0.0f, rest = 0.0f;
  int count = 0, tokens = 0;
  if (group < groups && e < a.E) {
    constexpr int U = 8;  // runs whose loads are in flight together
    for (int p = group; p < parts; p += groups * U) {
      uint32_t s[U], c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = p + u * groups < parts;
        const uint32_t* w = part_at(on ? p + u * groups : p);
        s[u] = on ? w[e] : 0u;
        c[u] = on ? w[a.E + e] : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        add_kept(sum, rest, __uint_as_float(s[u]));
        count += (int)c[u];
      }
    }
  }
  for (int p = threadIdx.x; p < parts; p += THREADS) tokens += (int)part_at(p)[2 * a.E];
  tokens = __reduce_add_sync(ALL, tokens);
  if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(&sh.tokens, tokens);
  sh.sums[threadIdx.x] = sum + rest;
  sh.counts[threadIdx.x] = count;
  __syncthreads();
  for (int h = 1 << (31 - __clz(max(groups - 1, 1))); h > 0; h >>= 1) {  // (from the largest power of two below)
    if (group < h && group + h < groups) {
      sh.sums[threadIdx.x] += sh.sums[threadIdx.x + h * width];
      sh.counts[threadIdx.x] += sh.counts[threadIdx.x + h * width];
    }
    __syncthreads();
  }
  const float n = (float)max(sh.tokens, 1);
  const float unit = a.coefficient * ((float)a.E / (float)a.K) / n;
  float term = 0.0f;
  if (group == 0 && e < a.E) {
    sum = sh.sums[threadIdx.x];
    count = sh.counts[threadIdx.x];
    a.counts[s * a.E + e] = count;
    const float slope = unit * (float)count / n;
    a.slope[s * a.E + e] = slope;
    term = slope * sum;
  }
  // (experts of a CTA: at most 64, so two warps hold terms)
  __syncthreads();
  sh.sums[threadIdx.x] = term;
  __syncthreads();
  if (threadIdx.x < 32) {
    float v = sh.sums[threadIdx.x] + sh.sums[threadIdx.x + 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
    if (threadIdx.x == 0) sh.loss = v;
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    float v = 0.0f;
    for (int r = 0; r < JOIN; ++r) v += *cluster.map_shared_rank(&sh.loss, r);
    if (a.sequences == 1)
      *a.loss = v;
    else {
      a.seq_loss[s] = v;
      a.seq_tokens[s] = sh.tokens;
    }
  }
  cluster.sync();  // (shared memory stays until every CTA has read it)
}

// Few rows of one sequence: one cluster, joined through distributed shared
// memory.
template <typename T, bool VEC, int C>
__global__ void __launch_bounds__(THREADS) balance_small_kernel(BalanceArgs a) {
  __shared__ SumShared sh;
  __shared__ SmallShared own;
  int64_t lo = 0, hi = a.rows;
  if (a.offsets) lo = bound_of(a, 0), hi = bound_of(a, 1);
  const int64_t share = (hi - lo + JOIN - 1) / JOIN;
  const int64_t begin = min(lo + blockIdx.x * share, hi), end = min(begin + share, hi);
  sum_run<T, VEC, C>(a, begin, max(begin, end), sh, own.part);
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  join_parts<THREADS>(a, 0, JOIN, [&](int p) { return (const uint32_t*)cluster.map_shared_rank(&own.part[0], p); },
                      own.join);
}

// A CTA sums its block of rows, run by run.
template <typename T, bool VEC, int C>
__global__ void __launch_bounds__(THREADS, C <= 2 ? 5 : C <= 4 ? 3 : 2) balance_sum_kernel(BalanceArgs a) {
  __shared__ SumShared sh;
  __shared__ Walk walk;
  pdl_trigger();
  const int64_t begin = min((int64_t)blockIdx.x * a.block_rows, a.rows);
  const int64_t end = min(begin + a.block_rows, a.rows);
  int64_t seq = walk.first(a, begin);
  for (int64_t at = begin; at < end;) {
    const Run r = walk.next(a, at, end, seq);
    // (a block and a sequence meet once: block + sequence numbers their runs)
    if (r.seq >= 0) sum_run<T, VEC, C>(a, r.lo, r.hi, sh, a.parts + (blockIdx.x + r.seq) * part_words(a.E));
    at = r.hi;
  }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) balance_join_kernel(BalanceArgs a) {
  __shared__ JoinShared<THREADS> sh;
  pdl_wait();
  pdl_trigger();
  const int64_t s = blockIdx.x / JOIN;
  int64_t first = 0;
  int parts = a.blocks;
  if (a.offsets) {
    const int64_t lo = bound_of(a, s), hi = bound_of(a, s + 1);
    first = hi > lo ? lo / a.block_rows : 0;
    parts = hi > lo ? (int)((hi - 1) / a.block_rows - first + 1) : 0;
  }
  const uint32_t* base = a.parts + (first + s) * part_words(a.E);
  join_parts<THREADS>(a, s, parts, [&](int p) { return base + (int64_t)p * part_words(a.E); }, sh);
}

// Several sequences: the mean over those with tokens.
__global__ void __launch_bounds__(THREADS) balance_mean_kernel(BalanceArgs a) {
  __shared__ float losses[THREADS];
  __shared__ int used;
  if (threadIdx.x == 0) used = 0;
  __syncthreads();
  pdl_wait();
  int n = 0;
  float loss = 0.0f, rest = 0.0f;
  for (int64_t s = threadIdx.x; s < a.sequences; s += THREADS) {
    n += a.seq_tokens[s] > 0;
    if (blockIdx.x == 0) add_kept(loss, rest, a.seq_loss[s]);
  }
  n = __reduce_add_sync(ALL, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&used, n);
  losses[threadIdx.x] = isfinite(loss) ? loss + rest : loss;
  __syncthreads();
  const float share = 1.0f / (float)max(used, 1);
  const int64_t all = a.sequences * a.E;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < all; i += (int64_t)gridDim.x * THREADS)
    a.slope[i] *= share;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    float v = 0.0f;
    for (int i = threadIdx.x; i < THREADS; i += 32) v += losses[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
    if (threadIdx.x == 0) *a.loss = v * share;
  }
}

// The gradient: with g = dloss * slope (of the row's sequence) and its mean
// under the shares, dl = p (g - mean), or s (1 - s) (g - mean) / sum for sigmoid
// scores; plus `add`.  A row is read by the lanes that write it, before they
// write, so dlogits may be logits or add.
template <typename T, bool VEC, int C>
__global__ void __launch_bounds__(THREADS, C <= 2 ? 3 : C <= 4 ? 2 : 1) balance_grad_kernel(BalanceArgs a) {
  using Part = RowPart<T, VEC, C>;
  constexpr int N = Part::N;
  __shared__ Walk walk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 15, half = lane >> 4;
  const int64_t begin = (int64_t)blockIdx.x * a.block_rows;
  const int64_t end = begin + a.block_rows < a.rows ? begin + a.block_rows : a.rows;
  const T* logits = static_cast<const T*>(a.logits);
  const T* add = static_cast<const T*>(a.add);
  T* dlogits = static_cast<T*>(a.dlogits);
  const float dloss = a.dloss ? *a.dloss : 1.0f;
  int64_t seq = walk.first(a, begin);
  for (int64_t at = begin; at < end;) {
    const Run run = walk.next(a, at, end, seq);
    at = run.hi;
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = Part::expert(i, sub);
      g[i] = run.seq >= 0 && e < a.E ? a.slope[run.seq * a.E + e] * dloss : 0.0f;
    }
    const auto fetch = [&](int64_t row, Part& p) {
      const bool in = row < run.hi && run.seq >= 0;
      const bool on = in && (!a.mask || a.mask[row]);
      p.load(logits + row * a.stride, a.E, sub, in, minus_infinity<T>());
      return on;
    };
    Part cur;
    bool on = fetch(run.lo + warp * 2 + half, cur);
    for (int64_t base = run.lo + warp * 2; base < run.hi; base += ROWS_AT_ONCE) {
      const int64_t row = base + half;
      // (add's own row as late as its registers allow: both prefetched spill)
      Part more, nxt;
      if (add) more.load(add + row * a.add_stride, a.E, sub, row < run.hi, 0u);
      const bool nxt_on = fetch(row + ROWS_AT_ONCE, nxt);
      float x[N];
      cur.values(x);
      float mean = 0.0f;
      if (a.sigmoid) {
        float rest[N];
        const float inv = sigmoid_scores<N, true>(x, rest);
#pragma unroll
        for (int i = 0; i < N; ++i) mean = fmaf(x[i], g[i], mean);
        mean = row_sum(mean) * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] * rest[i] * ((g[i] - mean) * inv);
      } else {
        const float inv = softmax_scores(x);
#pragma unroll
        for (int i = 0; i < N; ++i) mean = fmaf(x[i], g[i], mean);
        mean = row_sum(mean) * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] * inv * (g[i] - mean);
      }
      if (!on) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.0f;
      }
      if (add) {
        float y[N];
        more.values(y);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += y[i];
      }
      if (row < run.hi) Part::store(dlogits + row * a.dstride, a.E, sub, x);
      cur = nxt;
      on = nxt_on;
    }
  }
}

// ---- launches ----

cudaError_t launch(void (*kernel)(BalanceArgs), int64_t grid, int threads, int cluster, bool pdl, cudaStream_t s,
                   const BalanceArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim = {(unsigned)cluster, 1, 1};
    ++cfg.numAttrs;
  }
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

using Kernel = void (*)(BalanceArgs);
enum Which { SUM, SMALL, GRAD };

template <typename T, bool VEC, int C>
Kernel pick(Which w) {
  return w == SUM ? balance_sum_kernel<T, VEC, C> : w == SMALL ? balance_small_kernel<T, VEC, C> : balance_grad_kernel<T, VEC, C>;
}

template <typename T, bool VEC>
Kernel kernel_for(int E, Which w) {
  switch ((E + 63) / 64) {
    case 1: return pick<T, VEC, 1>(w);
    case 2: return pick<T, VEC, 2>(w);
    case 3: return pick<T, VEC, 3>(w);
    case 4: return pick<T, VEC, 4>(w);
  }
  return pick<T, VEC, 8>(w);
}

Kernel kernel_for(const BalanceArgs& a, bool vec, Which w) {
  if (a.dtype == MOE_DTYPE_F32) return vec ? kernel_for<float, true>(a.E, w) : kernel_for<float, false>(a.E, w);
  if (a.dtype == MOE_DTYPE_F16) return vec ? kernel_for<__half, true>(a.E, w) : kernel_for<__half, false>(a.E, w);
  return vec ? kernel_for<__nv_bfloat16, true>(a.E, w) : kernel_for<__nv_bfloat16, false>(a.E, w);
}

// CTAs of one wave: as many an SM as the kernels' registers allow.
int64_t sum_ctas(int E) { return 152 * (E <= 128 ? 5 : E <= 256 ? 3 : 2); }
int64_t grad_ctas(int E) { return 152 * (E <= 128 ? 3 : E <= 256 ? 2 : 1); }
// Logits that one cluster takes, in one launch (512 KB of FP32: eight SMs read
// that in the time that a second launch takes), of rows that its lanes add at once.
constexpr int64_t SMALL_ELEMENTS = 1 << 17, SMALL_ROWS = JOIN * SUM_ROWS;

int64_t rows_of_a_block(int64_t rows, int64_t ctas) {
  const int64_t r = (rows + ctas - 1) / ctas;
  return std::max<int64_t>((r + ROWS_AT_ONCE - 1) / ROWS_AT_ONCE * ROWS_AT_ONCE, ROWS_AT_ONCE);
}

// Rows of a CTA that sums: one wave of CTAs, or more where its runs would be too long.
int64_t rows_of_a_run(int E, int64_t rows) {
  return std::min<int64_t>(rows_of_a_block(rows, sum_ctas(E)), (E > 64 * LONG_RUNS ? 32 : 1) * SUM_ROWS);
}

int64_t sum_blocks(int E, int64_t rows) {
  const int64_t r = rows_of_a_run(E, rows);
  return (rows + r - 1) / r;
}

bool small_call(int E, int64_t rows, int64_t sequences) {
  return sequences == 1 && rows * E <= SMALL_ELEMENTS && rows <= SMALL_ROWS;
}

}  // namespace

size_t balance_workspace(int E, int64_t rows, int64_t sequences) {
  if (small_call(E, rows, sequences)) return 0;
  // (the runs' sums, then a loss and the tokens of each sequence)
  return ((size_t)(sum_blocks(E, rows) + sequences) * part_words(E) + 2 * (size_t)sequences) * 4;
}

cudaError_t launch_balance(BalanceArgs a, bool vec, void* workspace, cudaStream_t s) {
  if (small_call(a.E, a.rows, a.sequences)) return launch(kernel_for(a, vec, SMALL), JOIN, THREADS, JOIN, false, s, a);
  a.block_rows = rows_of_a_run(a.E, a.rows);
  const int64_t blocks = sum_blocks(a.E, a.rows);
  a.parts = static_cast<uint32_t*>(workspace);
  a.seq_loss = reinterpret_cast<float*>(a.parts + (blocks + a.sequences) * part_words(a.E));
  a.seq_tokens = reinterpret_cast<int32_t*>(a.seq_loss + a.sequences);
  cudaError_t e = cudaSuccess;
  a.blocks = (int)blocks;
  if (blocks) e = launch(kernel_for(a, vec, SUM), blocks, THREADS, 1, false, s, a);
  if (e != cudaSuccess) return e;
  const bool one = a.sequences == 1;
  e = launch(one ? balance_join_kernel<JOIN_THREADS> : balance_join_kernel<THREADS>, a.sequences * JOIN,
             one ? JOIN_THREADS : THREADS, JOIN, blocks > 0, s, a);
  if (e != cudaSuccess || a.sequences == 1) return e;
  const int64_t want = (a.sequences * a.E + THREADS * 4 - 1) / (THREADS * 4);
  return launch(balance_mean_kernel, std::min<int64_t>(want, 304), THREADS, 1, true, s, a);
}

cudaError_t launch_balance_backward(BalanceArgs a, bool vec, cudaStream_t s) {
  a.block_rows = rows_of_a_block(a.rows, grad_ctas(a.E));
  return launch(kernel_for(a, vec, GRAD), (a.rows + a.block_rows - 1) / a.block_rows, THREADS, 1, false, s, a);
}

}  // namespace moe
