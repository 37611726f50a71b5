// kernels_clip.cu - the norm of many gradients together, and their clipping.
//
// Two passes over the tensors, in chunks of 32 KB that a grid takes in turn: the
// first, one wave, leaves a sum of squares for each CTA (763 MB: 110 us, the rate
// of a copy), the second adds those up (in every CTA, in the same order) and
// scales (763 MB read, 763 written: 218 us, a copy's rate and what L2 spares).  Both
// are bound by bytes; the second goes through the chunks from the last to the first,
// so that what the first left in L2 need not come from memory again.  Sets of a
// few chunks are one launch of one cluster.
//
// (One launch each, caches flushed: 216 quiet tensors, 48 MB, 12 us for the norm and 8
// for the pass that finds nothing to do, the two 12.6 together where the set stays in
// L2; 14 tensors, 135 KB, one cluster: 10.)
//
// The list of tensors travels as a kernel parameter: no copy to the device, no
// buffer of addresses that a captured graph would have to keep.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "elem_types.cuh"
#include "kernels_ops.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int GRANULES = 8;                    // 16-byte granules a thread and chunk
constexpr int CHUNK = THREADS * GRANULES;      // granules of a chunk
constexpr int SMALL_CTAS = 8;                  // the cluster of a small set
constexpr uint32_t SMALL_CHUNKS = 32;
constexpr int SCALE_WAVES = 12;                // of the scaling grid: 382 M bf16 values, clipped,
                                               // 352 us; one wave 364, 40 waves 355
constexpr unsigned ALL = 0xffffffffu;

// Tensors of one launch, and the number of their first chunks.
template <int CAP>
struct List {
  const void* src[CAP];
  void* dst[CAP];
  int64_t count[CAP];
  uint32_t first[CAP + 1];
  uint8_t dtype[CAP];
  int n;
  double* sums;       // of the grid's CTAs
  int parts;          // CTAs that leave a sum
  bool add;           // onto the sums that are there (a set of several lists)
  float* norm;
  float limit, eps;
  bool scale;         // (of a small set: more than the norm)
  bool in_place;      // every tensor
};

// Chunk `id` of a list: the tensor's data from the 16-byte granule it starts
// in, and which of its elements count.
struct Chunk {
  int tensor, dtype;
  int64_t granule;    // first one, from the tensor's first
};

template <int CAP>
__device__ __forceinline__ Chunk chunk_of(const List<CAP>& l, uint32_t id) {
  int lo = 0, hi = l.n - 1;  // the last tensor whose first chunk is at or before id
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= id)
      lo = mid;
    else
      hi = mid - 1;
  }
  return {lo, l.dtype[lo], (int64_t)(id - l.first[lo]) * CHUNK};
}

// A thread's granules of a chunk: whole ones by one load, those that the
// tensor's ends cut element by element (zeros outside).
template <typename T>
struct Granules {
  static constexpr int N = 16 / sizeof(T);
  uint4 q[GRANULES];
  __device__ __forceinline__ static int head(const void* p) { return (int)((uintptr_t)p & 15) / (int)sizeof(T); }
  __device__ __forceinline__ void load(const void* src, int64_t count, int64_t granule) {
    const int h = head(src);
    const T* base = static_cast<const T*>(src) - h;
#pragma unroll
    for (int j = 0; j < GRANULES; ++j) {
      const int64_t at = (granule + j * THREADS + threadIdx.x) * N;
      q[j] = make_uint4(0, 0, 0, 0);
      if (at >= h && at + N <= h + count) {
        q[j] = *reinterpret_cast<const uint4*>(base + at);
      } else if (at + N > h && at < h + count) {
        T* e = reinterpret_cast<T*>(&q[j]);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at + i >= h && at + i < h + count) e[i] = base[at + i];
      }
    }
  }
  // dst starts at the same offset from a 16-byte boundary, or is written
  // element by element.
  __device__ __forceinline__ void store_scaled(const void* src, void* dst, int64_t count, int64_t granule,
                                               float f) const {
    const int h = head(src);
    T* base = static_cast<T*>(dst) - h;
    const bool whole = ((uintptr_t)base & 15) == 0;
#pragma unroll
    for (int j = 0; j < GRANULES; ++j) {
      const int64_t at = (granule + j * THREADS + threadIdx.x) * N;
      if (at + N <= h || at >= h + count) continue;
      uint4 o;
      const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          r[i] = __float_as_uint(__uint_as_float(w[i]) * f);
        } else {
          const float2 v = unpack2(w[i], T());
          r[i] = pack2(v.x * f, v.y * f, T());
        }
      }
      o = make_uint4(r[0], r[1], r[2], r[3]);
      if (whole && at >= h && at + N <= h + count) {
        *reinterpret_cast<uint4*>(base + at) = o;
      } else {
        const T* e = reinterpret_cast<const T*>(&o);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at + i >= h && at + i < h + count) base[at + i] = e[i];
      }
    }
  }
  __device__ __forceinline__ float squares() const {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < GRANULES; ++j) {
      const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          const float v = __uint_as_float(w[i]);
          s[i & 1] = fmaf(v, v, s[i & 1]);
        } else {
          const float2 v = unpack2(w[i], T());
          s[0] = fmaf(v.x, v.x, s[0]);
          s[1] = fmaf(v.y, v.y, s[1]);
        }
      }
    }
    return s[0] + s[1];
  }
  __device__ __forceinline__ bool zero() const {
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < GRANULES; ++j) any |= q[j].x | q[j].y | q[j].z | q[j].w;
    return (any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0;
  }
  __device__ __noinline__ static double squares_wide(const uint4* q) {
    double s = 0.0;
    for (int j = 0; j < GRANULES; ++j) {
      const T* e = reinterpret_cast<const T*>(q + j);
      for (int i = 0; i < N; ++i) {
        const double v = (double)to_f32(e[i]);
        s += v * v;
      }
    }
    return s;
  }
};

// A thread's sum of squares: FP32 for chunks whose squares keep their bits
// there, FP64 for the rest (some hundred times slower, so only where a sum of
// 64 squares leaves [2^-90, 2^100]).  What an FP32 addition of a chunk rounds away is
// kept (add_kept) and added at the end: a large set gives a thread hundreds of
// chunks, whose roundings, of gradients alike, would all go one way (862 chunks: 66
// units of 2^-24 in the norm).
struct Squares {
  float sum = 0.0f, rest = 0.0f;
  double wide = 0.0;
  template <typename T>
  __device__ __forceinline__ void add(const Granules<T>& g) {
    const float s = g.squares();
    if (s > 0x1p-90f && s < 0x1p100f)
      add_kept(sum, rest, s);
    else if (!g.zero()) {
      uint4 q[GRANULES];
#pragma unroll
      for (int j = 0; j < GRANULES; ++j) q[j] = g.q[j];
      wide += Granules<T>::squares_wide(q);
    }
  }
};

template <int CAP>
__device__ __forceinline__ void add_chunk(const List<CAP>& l, uint32_t id, Squares& s) {
  const Chunk c = chunk_of(l, id);
  if (c.dtype == MOE_DTYPE_F32) {
    Granules<float> g;
    g.load(l.src[c.tensor], l.count[c.tensor], c.granule);
    s.add(g);
  } else if (c.dtype == MOE_DTYPE_F16) {
    Granules<__half> g;
    g.load(l.src[c.tensor], l.count[c.tensor], c.granule);
    s.add(g);
  } else {
    Granules<__nv_bfloat16> g;
    g.load(l.src[c.tensor], l.count[c.tensor], c.granule);
    s.add(g);
  }
}

template <typename T, int CAP>
__device__ __forceinline__ void scale_typed(const List<CAP>& l, const Chunk& c, float f) {
  Granules<T> g;
  g.load(l.src[c.tensor], l.count[c.tensor], c.granule);
  g.store_scaled(l.src[c.tensor], l.dst[c.tensor], l.count[c.tensor], c.granule, f);
}
template <int CAP>
__device__ __forceinline__ void scale_chunk(const List<CAP>& l, uint32_t id, float f) {
  const Chunk c = chunk_of(l, id);
  if (f == 1.0f && l.src[c.tensor] == l.dst[c.tensor]) return;  // nothing to change
  if (c.dtype == MOE_DTYPE_F32)
    scale_typed<float>(l, c, f);
  else if (c.dtype == MOE_DTYPE_F16)
    scale_typed<__half>(l, c, f);
  else
    scale_typed<__nv_bfloat16>(l, c, f);
}

// Over the CTA, the same in every thread (red: of THREADS / 32 values).
template <typename V>
__device__ __forceinline__ V block_sum(V v, double* red) {
  V* r = reinterpret_cast<V*>(red);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) t += r[w];
  __syncthreads();
  return t;
}

// The threads' sums: in FP32, which is four times as quick as FP64's shuffles
// and slow adds (its 13 steps round the sum by 2^-24 each), what they rounded away
// where a thread has several chunks, and FP64 only where a thread has some.
__device__ __forceinline__ double block_squares(const Squares& s, double* red) {
  double t = block_sum(s.sum, red);
  if (__syncthreads_or(s.rest != 0.0f)) t += (double)block_sum(s.rest, red);
  if (__syncthreads_or(s.wide != 0.0)) t += block_sum(s.wide, red);
  return t;
}

// Rounded once more than the FP64 root where the sum is an FP32 normal number.
__device__ __forceinline__ float root(double sum) {
  const float s = (float)sum;
  return s > 0x1p-120f && s < 0x1p126f ? sqrtf(s) : (float)sqrt(sum);
}

// min(1, limit / (norm + eps)); NaN where the norm is.
__device__ __forceinline__ float factor(float norm, float limit, float eps) {
  const float f = limit / (norm + eps);
  return f >= 1.0f ? 1.0f : f;
}

template <int CAP>
__global__ void __launch_bounds__(THREADS) gradient_squares_kernel(const __grid_constant__ List<CAP> l) {
  __shared__ double red[THREADS / 32];
  pdl_trigger();
  Squares s;
  const uint32_t chunks = l.first[l.n];
  for (uint32_t id = blockIdx.x; id < chunks; id += gridDim.x) add_chunk(l, id, s);
  const double t = block_squares(s, red);
  if (threadIdx.x == 0) l.sums[blockIdx.x] = l.add ? l.sums[blockIdx.x] + t : t;
}

__device__ __forceinline__ float norm_of(const double* sums, int parts, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += THREADS) v += sums[i];
  return root(block_sum(v, red));
}

template <int CAP>
__global__ void __launch_bounds__(THREADS) gradient_scale_kernel(const __grid_constant__ List<CAP> l) {
  __shared__ double red[THREADS / 32];
  pdl_wait();
  const float norm = norm_of(l.sums, l.parts, red);
  if (blockIdx.x == 0 && threadIdx.x == 0) *l.norm = norm;
  const float f = factor(norm, l.limit, l.eps);
  if (f == 1.0f && l.in_place) return;
  const uint32_t chunks = l.first[l.n];
  for (uint32_t id = blockIdx.x; id < chunks; id += gridDim.x) scale_chunk(l, chunks - 1 - id, f);
}

__global__ void __launch_bounds__(THREADS) gradient_norm_kernel(const double* sums, int parts, float* norm) {
  __shared__ double red[THREADS / 32];
  pdl_wait();
  const float v = norm_of(sums, parts, red);
  if (threadIdx.x == 0) *norm = v;
}

// One cluster: its CTAs' sums meet in shared memory.
template <int CAP>
__global__ void __launch_bounds__(THREADS) gradient_small_kernel(const __grid_constant__ List<CAP> l) {
  __shared__ double red[THREADS / 32];
  __shared__ double mine;
  cg::cluster_group cluster = cg::this_cluster();
  Squares s;
  const uint32_t chunks = l.first[l.n];
  for (uint32_t id = blockIdx.x; id < chunks; id += SMALL_CTAS) add_chunk(l, id, s);
  const double t = block_squares(s, red);
  if (threadIdx.x == 0) mine = t;
  cluster.sync();
  double all = 0.0;
  for (int r = 0; r < SMALL_CTAS; ++r) all += *cluster.map_shared_rank(&mine, r);
  const float norm = root(all);
  if (blockIdx.x == 0 && threadIdx.x == 0) *l.norm = norm;
  if (l.scale) {
    const float f = factor(norm, l.limit, l.eps);
    for (uint32_t id = blockIdx.x; id < chunks; id += SMALL_CTAS) scale_chunk(l, id, f);
  }
  cluster.sync();  // (shared memory stays until every CTA has read it)
}

constexpr int FEW = 64, SOME = 256, MANY = 1024;  // tensors of a launch: 2, 8 or 30 KB of parameters
static_assert(sizeof(List<MANY>) <= 32764, "kernel parameters");

uint32_t chunks_of(const moe_gradient& t) {
  const int64_t b = t.dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (t.count == 0) return 0;
  const int64_t bytes = (int64_t)((uintptr_t)t.data & 15) + t.count * b;
  return (uint32_t)((bytes + 16 * CHUNK - 1) / (16 * CHUNK));
}

template <int CAP>
void fill(List<CAP>& l, const moe_gradient* t, int n) {
  uint32_t at = 0;
  l.in_place = true;
  for (int i = 0; i < n; ++i) {
    l.in_place = l.in_place && t[i].data == t[i].out;
    l.src[i] = t[i].data;
    l.dst[i] = t[i].out;
    l.count[i] = t[i].count;
    l.dtype[i] = (uint8_t)t[i].dtype;
    l.first[i] = at;
    at += chunks_of(t[i]);
  }
  l.first[n] = at;
  l.n = n;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(SMALL_CTAS);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {SMALL_CTAS, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int CAP>
cudaError_t run(const moe_gradient* t, int64_t n, const ClipArgs& a, cudaStream_t s) {
  List<CAP> l;
  uint32_t most = 0;
  for (int64_t i = 0; i < n; i += CAP) {
    uint32_t c = 0;
    for (int64_t j = i; j < std::min<int64_t>(n, i + CAP); ++j) c += chunks_of(t[j]);
    most = std::max(most, c);
  }
  l.norm = a.norm;
  l.limit = a.limit;
  l.eps = a.eps;
  l.scale = a.scale;
  l.sums = a.sums;
  l.add = false;
  l.parts = (int)std::min<uint32_t>(std::max<uint32_t>(most, 1), CLIP_PARTS);
  if (n <= CAP && most <= SMALL_CHUNKS) {
    fill(l, t, (int)n);
    return launch_cluster(gradient_small_kernel<CAP>, s, l);
  }
  for (int64_t i = 0; i < n; i += CAP) {
    fill(l, t + i, (int)std::min<int64_t>(n - i, CAP));
    l.add = i > 0;
    const cudaError_t e = launch_k(gradient_squares_kernel<CAP>, dim3(l.parts), dim3(THREADS), 0, s, false, l);
    if (e != cudaSuccess) return e;
  }
  if (!a.scale)
    return launch_k(gradient_norm_kernel, dim3(1), dim3(THREADS), 0, s, true, (const double*)a.sums, l.parts, a.norm);
  for (int64_t i = 0; i < n; i += CAP) {
    if (n > CAP) fill(l, t + i, (int)std::min<int64_t>(n - i, CAP));
    // (in place one wave: most steps change nothing, and its CTAs only look: 48 MB
    // in 216 tensors, caches flushed, both passes and two events 24 us, with twelve
    // waves 32)
    const uint32_t grid = std::min<uint32_t>(l.first[l.n], (l.in_place ? 1 : SCALE_WAVES) * CLIP_PARTS);
    const cudaError_t e =
        launch_k(gradient_scale_kernel<CAP>, dim3(std::max(grid, 1u)), dim3(THREADS), 0, s, n <= CAP, l);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_clip(const moe_gradient* t, int64_t n, const ClipArgs& a, cudaStream_t s) {
  return n <= FEW ? run<FEW>(t, n, a, s) : n <= SOME ? run<SOME>(t, n, a, s) : run<MANY>(t, n, a, s);
}

}  // namespace moe
