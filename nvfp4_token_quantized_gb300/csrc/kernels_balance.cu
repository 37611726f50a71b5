// kernels_balance.cu - the balance loss of the expert choice, the counts of
// the chosen experts, and the loss's gradient.
//
// A token's shares p are its softmax, or its sigmoid scores over their sum.
// The loss of a sequence of N tokens is coefficient * E / (K N^2) times the sum
// over the experts of (times chosen) * (sum of p), so one pass over the logits
// leaves E sums and E counts a run of rows, which a second, small kernel joins
// in the order of the runs: no atomics on floats, the same bits every time.
//
// Sixteen lanes share a row: four experts a lane and chunk, so that a row of
// 256 takes four 16-byte loads a lane and two trees of four steps for a
// maximum and a sum, and the lanes' own sums over the rows stay in registers.
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
constexpr int JOIN = 8;                  // CTAs of a cluster that joins the runs' sums
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

// x becomes scores that are the shares times their sum; returns 1 / sum, 0
// for a row of closed experts.  The hardware's exponential and quotient (some
// 2^-22 of a score; the logits' distance from the maximum times 2^-24 more).
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
    x[i] = __expf(x[i] - m);
    total += x[i];
  }
  total = row_sum(total);
  return total == 0.0f ? 0.0f : __fdividef(1.0f, total);
}
// The same for sigmoid scores, with the sum's own 1e-20; rest, if wanted, gets
// 1 - s, without the cancellation.
template <int N, bool REST>
__device__ __forceinline__ float sigmoid_scores(float (&x)[N], float (&rest)[REST ? N : 1]) {
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = __expf(-fabsf(x[i]));
    const float r = __fdividef(1.0f, 1.0f + a);
    const bool up = x[i] >= 0.0f;
    if constexpr (REST) rest[i] = up ? a * r : r;
    x[i] = up ? r : a * r;
    total += x[i];
  }
  return __fdividef(1.0f, row_sum(total) + SELECT_SUM_EPS);
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

// The sequence that row `row` lies in or before (block-wide: a count of the
// ends at or before it).
__device__ __forceinline__ int64_t first_sequence(const BalanceArgs& a, int64_t row, int* count) {
  if (!a.offsets) return 0;
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  int n = 0;
  for (int64_t i = threadIdx.x; i < a.sequences; i += THREADS) n += bound_of(a, i + 1) <= row;
  n = __reduce_add_sync(ALL, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(count, n);
  __syncthreads();
  return *count;
}

// The run that starts at row `at` < end; seq moves on to its sequence.  It
// ends behind `at` whatever the offsets hold.
__device__ __forceinline__ Run next_run(const BalanceArgs& a, int64_t at, int64_t end, int64_t& seq) {
  if (!a.offsets) return {at, end, 0};
  while (seq < a.sequences && bound_of(a, seq + 1) <= at) ++seq;
  if (seq >= a.sequences) return {at, end, -1};
  const int64_t lo = bound_of(a, seq), hi = bound_of(a, seq + 1);
  if (at < lo) return {at, lo < end ? lo : end, -1};
  return {at, hi < end ? hi : end, seq};
}

// Words of a run's sums: E sums of shares, E counts, the tokens.
__host__ __device__ __forceinline__ int part_words(int E) { return 2 * E + 1; }

struct SumShared {
  float sums[WARPS][SELECT_MAX_EXPERTS];
  int counts[SELECT_MAX_EXPERTS];
  int tokens, sequence;
  uint32_t part[2 * SELECT_MAX_EXPERTS + 1];  // (of a cluster that joins its own)
  float join_sum[THREADS];
  int join_count[THREADS];
  float loss;
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
  const auto fetch = [&](int64_t row, Part& p) {
    const bool on = row < hi && (!a.mask || a.mask[row]);
    p.load(logits + row * a.stride, a.E, sub, on, minus_infinity<T>());
    return on;
  };
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  int mine = 0;
  Part cur;
  bool on = fetch(lo + warp * 2 + half, cur);

  // (the chosen experts while the first rows are on their way)
  const uint32_t slots = (uint32_t)((hi - lo) * a.K);
  const int32_t* ids = a.ids + lo * a.K;
  for (uint32_t i = threadIdx.x; i < slots; i += THREADS) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)a.E && (!a.mask || a.mask[lo + i / (uint32_t)a.K])) atomicAdd(&sh.counts[id], 1);
  }

  for (int64_t base = lo + warp * 2; base < hi; base += ROWS_AT_ONCE) {
    Part nxt;
    const bool nxt_on = fetch(base + ROWS_AT_ONCE + half, nxt);
    float x[N];
    cur.values(x);
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
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    acc[i] += __shfl_xor_sync(ALL, acc[i], 16);
    const int e = Part::expert(i, sub);
    if (half == 0 && e < a.E) sh.sums[warp][e] = acc[i];
  }
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
template <typename PartAt>
__device__ __forceinline__ void join_parts(const BalanceArgs& a, int64_t s, int parts, PartAt part_at, SumShared& sh) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int width = (a.E + JOIN - 1) / JOIN, groups = THREADS / width;
  const int local = threadIdx.x % width, group = threadIdx.x / width, e = rank * width + local;
  if (threadIdx.x == 0) sh.tokens = 0;
  __syncthreads();
  float sum = 0.0f;
  int count = 0, tokens = 0;
  if (group < groups && e < a.E) {
#pragma unroll 4
    for (int p = group; p < parts; p += groups) {
      const uint32_t* w = part_at(p);
      sum += __uint_as_float(w[e]);
      count += (int)w[a.E + e];
    }
  }
  for (int p = threadIdx.x; p < parts; p += THREADS) tokens += (int)part_at(p)[2 * a.E];
  tokens = __reduce_add_sync(ALL, tokens);
  if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(&sh.tokens, tokens);
  sh.join_sum[threadIdx.x] = sum;
  sh.join_count[threadIdx.x] = count;
  __syncthreads();
  const float n = (float)max(sh.tokens, 1);
  const float unit = a.coefficient * ((float)a.E / (float)a.K) / n;
  float term = 0.0f;
  if (group == 0 && e < a.E) {
    for (int g = 1; g < groups; ++g) {
      sum += sh.join_sum[g * width + local];
      count += sh.join_count[g * width + local];
    }
    a.counts[s * a.E + e] = count;
    const float slope = unit * (float)count / n;
    a.slope[s * a.E + e] = slope;
    term = slope * sum;
  }
  // (experts of a CTA: at most 64, so two warps hold terms)
  __syncthreads();
  sh.join_sum[threadIdx.x] = term;
  __syncthreads();
  if (threadIdx.x < 32) {
    float v = sh.join_sum[threadIdx.x] + sh.join_sum[threadIdx.x + 32];
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

// A CTA sums its block of rows, run by run.  One cluster alone joins its own
// sums through distributed shared memory.
template <typename T, bool VEC, int C>
__global__ void __launch_bounds__(THREADS) balance_sum_kernel(BalanceArgs a) {
  __shared__ SumShared sh;
  pdl_trigger();
  const int64_t begin = (int64_t)blockIdx.x * a.block_rows;
  const int64_t end = begin + a.block_rows < a.rows ? begin + a.block_rows : a.rows;
  if (a.small) {
    sum_run<T, VEC, C>(a, begin, end > begin ? end : begin, sh, sh.part);
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    join_parts(a, 0, JOIN, [&](int p) { return (const uint32_t*)cluster.map_shared_rank(&sh.part[0], p); }, sh);
    return;
  }
  int64_t seq = first_sequence(a, begin, &sh.sequence);
  for (int64_t at = begin; at < end;) {
    const Run r = next_run(a, at, end, seq);
    // (a block and a sequence meet once: block + sequence numbers their runs)
    if (r.seq >= 0) sum_run<T, VEC, C>(a, r.lo, r.hi, sh, a.parts + (blockIdx.x + r.seq) * part_words(a.E));
    at = r.hi;
  }
}

__global__ void __launch_bounds__(THREADS) balance_join_kernel(BalanceArgs a) {
  __shared__ SumShared sh;
  pdl_wait();
  pdl_trigger();
  const int64_t s = blockIdx.x / JOIN;
  int64_t lo = 0, hi = a.rows;
  if (a.offsets) lo = bound_of(a, s), hi = bound_of(a, s + 1);
  const int64_t first = hi > lo ? lo / a.block_rows : 0;
  const int parts = hi > lo ? (int)((hi - 1) / a.block_rows - first + 1) : 0;
  const uint32_t* base = a.parts + (first + s) * part_words(a.E);
  join_parts(a, s, parts, [&](int p) { return base + (int64_t)p * part_words(a.E); }, sh);
}

// Several sequences: the mean over those with tokens.
__global__ void __launch_bounds__(THREADS) balance_mean_kernel(BalanceArgs a) {
  __shared__ float losses[THREADS];
  __shared__ int used;
  if (threadIdx.x == 0) used = 0;
  __syncthreads();
  pdl_wait();
  int n = 0;
  float loss = 0.0f;
  for (int64_t s = threadIdx.x; s < a.sequences; s += THREADS) {
    n += a.seq_tokens[s] > 0;
    if (blockIdx.x == 0) loss += a.seq_loss[s];
  }
  n = __reduce_add_sync(ALL, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&used, n);
  losses[threadIdx.x] = loss;
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
__global__ void __launch_bounds__(THREADS) balance_grad_kernel(BalanceArgs a) {
  using Part = RowPart<T, VEC, C>;
  constexpr int N = Part::N;
  __shared__ int sequence;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 15, half = lane >> 4;
  const int64_t begin = (int64_t)blockIdx.x * a.block_rows;
  const int64_t end = begin + a.block_rows < a.rows ? begin + a.block_rows : a.rows;
  const T* logits = static_cast<const T*>(a.logits);
  const T* add = static_cast<const T*>(a.add);
  T* dlogits = static_cast<T*>(a.dlogits);
  const float dloss = a.dloss ? *a.dloss : 1.0f;
  int64_t seq = first_sequence(a, begin, &sequence);
  for (int64_t at = begin; at < end;) {
    const Run run = next_run(a, at, end, seq);
    at = run.hi;
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = Part::expert(i, sub);
      g[i] = run.seq >= 0 && e < a.E ? a.slope[run.seq * a.E + e] * dloss : 0.0f;
    }
    const auto fetch = [&](int64_t row, Part& p, Part& more) {
      const bool in = row < run.hi, on = in && run.seq >= 0 && (!a.mask || a.mask[row]);
      p.load(logits + row * a.stride, a.E, sub, on, minus_infinity<T>());
      if (add) more.load(add + row * a.add_stride, a.E, sub, in, 0u);
      return on;
    };
    Part cur, cur_add;
    bool on = fetch(run.lo + warp * 2 + half, cur, cur_add);
    for (int64_t base = run.lo + warp * 2; base < run.hi; base += ROWS_AT_ONCE) {
      Part nxt, nxt_add;
      const bool nxt_on = fetch(base + ROWS_AT_ONCE + half, nxt, nxt_add);
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
        cur_add.values(y);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += y[i];
      }
      const int64_t row = base + half;
      if (row < run.hi) Part::store(dlogits + row * a.dstride, a.E, sub, x);
      cur = nxt;
      cur_add = nxt_add;
      on = nxt_on;
    }
  }
}

// ---- launches ----

cudaError_t launch(void (*kernel)(BalanceArgs), int64_t grid, int cluster, bool pdl, cudaStream_t s,
                   const BalanceArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(THREADS);
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

template <typename T, bool VEC>
Kernel kernel_for(int E, bool grad) {
  switch ((E + 63) / 64) {
    case 1: return grad ? balance_grad_kernel<T, VEC, 1> : balance_sum_kernel<T, VEC, 1>;
    case 2: return grad ? balance_grad_kernel<T, VEC, 2> : balance_sum_kernel<T, VEC, 2>;
    case 3: return grad ? balance_grad_kernel<T, VEC, 3> : balance_sum_kernel<T, VEC, 3>;
    case 4: return grad ? balance_grad_kernel<T, VEC, 4> : balance_sum_kernel<T, VEC, 4>;
  }
  return grad ? balance_grad_kernel<T, VEC, 8> : balance_sum_kernel<T, VEC, 8>;
}

Kernel kernel_for(const BalanceArgs& a, bool vec, bool grad) {
  if (a.dtype == MOE_DTYPE_F32) return vec ? kernel_for<float, true>(a.E, grad) : kernel_for<float, false>(a.E, grad);
  if (a.dtype == MOE_DTYPE_F16)
    return vec ? kernel_for<__half, true>(a.E, grad) : kernel_for<__half, false>(a.E, grad);
  return vec ? kernel_for<__nv_bfloat16, true>(a.E, grad) : kernel_for<__nv_bfloat16, false>(a.E, grad);
}

constexpr int64_t SUM_CTAS = 152 * 2;     // one wave of two CTAs an SM
constexpr int64_t GRAD_CTAS = 152 * 2;
constexpr int64_t SMALL_ELEMENTS = 1 << 17;  // logits that one cluster takes

int64_t rows_of_a_block(int64_t rows, int64_t ctas) {
  const int64_t r = (rows + ctas - 1) / ctas;
  return std::max<int64_t>((r + ROWS_AT_ONCE - 1) / ROWS_AT_ONCE * ROWS_AT_ONCE, ROWS_AT_ONCE);
}

int64_t sum_blocks(int64_t rows) {
  const int64_t r = rows_of_a_block(rows, SUM_CTAS);
  return (rows + r - 1) / r;
}

bool small_call(int E, int64_t rows, bool offsets) { return !offsets && rows * E <= SMALL_ELEMENTS; }

}  // namespace

size_t balance_workspace(int E, int64_t rows, int64_t sequences) {
  // (the runs' sums, then a loss and the tokens of each sequence)
  return ((size_t)(sum_blocks(rows) + sequences) * part_words(E) + 2 * (size_t)sequences) * 4;
}

cudaError_t launch_balance(BalanceArgs a, bool vec, void* workspace, cudaStream_t s) {
  const Kernel sum = kernel_for(a, vec, false);
  if (small_call(a.E, a.rows, a.offsets != nullptr)) {
    a.small = true;
    a.block_rows = std::max<int64_t>((a.rows + JOIN - 1) / JOIN, 1);
    return launch(sum, JOIN, JOIN, false, s, a);
  }
  a.block_rows = rows_of_a_block(a.rows, SUM_CTAS);
  const int64_t blocks = sum_blocks(a.rows);
  a.parts = static_cast<uint32_t*>(workspace);
  a.seq_loss = reinterpret_cast<float*>(a.parts + (blocks + a.sequences) * part_words(a.E));
  a.seq_tokens = reinterpret_cast<int32_t*>(a.seq_loss + a.sequences);
  cudaError_t e = cudaSuccess;
  if (blocks) e = launch(sum, blocks, 1, false, s, a);
  if (e != cudaSuccess) return e;
  e = launch(balance_join_kernel, a.sequences * JOIN, JOIN, blocks > 0, s, a);
  if (e != cudaSuccess || a.sequences == 1) return e;
  const int64_t want = (a.sequences * a.E + THREADS * 4 - 1) / (THREADS * 4);
  return launch(balance_mean_kernel, std::min<int64_t>(want, 304), 1, true, s, a);
}

cudaError_t launch_balance_backward(BalanceArgs a, bool vec, cudaStream_t s) {
  a.block_rows = rows_of_a_block(a.rows, GRAD_CTAS);
  return launch(kernel_for(a, vec, true), (a.rows + a.block_rows - 1) / a.block_rows, 1, false, s, a);
}

}  // namespace moe
