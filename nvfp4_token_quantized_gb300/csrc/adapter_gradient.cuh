// adapter_gradient.cuh - the gradients of an adapter's factors, sums over its rows
// of hidden[row] (as a column) times x[row] (as a row), on the tensor cores' tcgen05
// path: D = x^T hidden, 128 columns of x by the ranks, contraction over the rows.
//
// Both operands lie as they are stored, rows of neighbouring columns, which is the
// layout of operands whose contraction runs across rows.  x's rows come by
// asynchronous copies of 512 bytes a row.  hidden is first split into its two
// 16-bit parts, by a kernel that writes them in the order and swizzle in which the
// tensor cores read them, once for all columns.  With FP16 the parts of one rank in a
// piece share a power of two: a rank's sums are a column of D of their own, so ranks
// of any size beside each other keep their bits.  (The search for the largest value
// of each rank: 16 us of 144 at 16384 rows of 32 ranks, under 1 of 20 at 777 of 8.)
//
// Rows that do not start on 16 bytes come as in adapter_tensor.cuh.  The CTAs' FP32
// sums are joined by a last kernel in the order of the rows.
//
// A CTA takes a piece (up to `unit` rows of one adapter) and 256 columns.  Bound by
// the bytes of x and dout, once each: 16384 rows of 4096 and 4096 columns, rank 32,
// 53 us (268 MB, 5.1 TB/s: two waves of CTAs, each with a start and an end), the
// split before 6 and the join behind 7.
#pragma once

#include <algorithm>

#include "adapter_mma.cuh"

namespace moe {

constexpr int GRADIENT_COLUMNS = 256;                      // of a CTA
constexpr int SPLIT_ROWS = 64;                             // of a CTA that splits

template <int R>
struct GradientShared {
  static constexpr int PANEL = GRADIENT_ROWS * 128;           // 64 columns of a stage's rows
  static constexpr int PARTS = 2 * R <= 64 ? 1 : 2 * R / 64;  // panels of hidden's two parts
  static constexpr int N = 2 * R < 64 ? 2 * R : 64;           // columns of one product
  static constexpr int X = GRADIENT_COLUMNS / 64 * PANEL, HIDDEN = PARTS * PANEL, STAGE = X + HIDDEN;
  static constexpr int STAGES = 4;
  static constexpr int D = R <= 64 ? 64 : 128;                // tensor memory columns of 128 columns of x
  static constexpr int BYTES = STAGES * STAGE + 1024;         // (aligned inside)
};

__device__ __forceinline__ int adapter_of(const OuterArgs& a, int group) {
  return a.group_of ? a.group_of[group] : group;
}

// Where a piece's stages of hidden's parts begin (numbered as pieces are), and
// where the sums of a group that begins at row `start` of the list and has several
// pieces: such a group of n rows has at most 2n / unit, so twice as many places as
// pieces of all rows are enough, whatever the number of adapters.
__device__ __forceinline__ int64_t first_stage(const Piece& p, int unit) {
  return (p.start - p.number * unit) / GRADIENT_ROWS + p.group + (int64_t)p.number * (unit / GRADIENT_ROWS);
}
__device__ __forceinline__ int64_t first_sums(int start, int unit) { return 2 * (int64_t)start / unit; }

// hidden's parts of one piece: [stage][panel][row] of 128 bytes, swizzled; ranks
// [0, R) of the panels' columns hold the first parts, [R, 2R) the second.
template <typename T, int R>
__global__ void __launch_bounds__(256) adapter_split_kernel(const OuterArgs a) {
  using S = GradientShared<R>;
  constexpr bool SCALED = !std::is_same<T, __nv_bfloat16>::value;
  __shared__ Piece found;
  __shared__ float some_max[SCALED ? 256 : 1], scale_of[SCALED ? R : 1];
  const int tid = threadIdx.x, side = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  // (blockIdx.z: SPLIT_ROWS of the piece's rows)
  const Piece p = find_piece(a.starts, a.rows, a.groups, a.unit, blockIdx.x, &found);
  if (p.group < 0 || adapter_of(a, p.group) == a.L) return;
  const float* hidden = a.hidden[side];
  const int32_t* rows = a.row_list + p.start;
  constexpr int G = R / 8;  // threads of a row, eight ranks each
  const int lane8 = tid % G;
  const auto load = [&](int r, float (&v)[8]) {
    const float* h = hidden + (r < p.count ? (int64_t)rows[r] * a.rank : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r < p.count && lane8 * 8 + i < a.rank ? h[lane8 * 8 + i] : 0.0f;
  };
  if constexpr (SCALED) {  // the largest value of each rank
    const int rank = tid % R;
    float m = 0.0f;
    if (rank < a.rank) {
      constexpr int U = 8, STEP = 256 / R;  // rows whose loads are in flight together
      for (int r = tid / R; r < p.count; r += U * STEP) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          v[u] = r + u * STEP < p.count ? hidden[(int64_t)rows[r + u * STEP] * a.rank + rank] : 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) m = fmaxf(m, fabsf(v[u]));
      }
    }
    some_max[tid] = m;
    __syncthreads();
    if (tid < R) {
#pragma unroll
      for (int w = R; w < 256; w += R) m = fmaxf(m, some_max[w + tid]);
      float back;
      scale_of[tid] = exponent_scale(m, back);
      if (blockIdx.z == 0 && tid < a.rank) a.back[side][(int64_t)blockIdx.x * a.rank + tid] = back;
    }
    __syncthreads();
  }
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = SCALED ? scale_of[lane8 * 8 + i] : 1.0f;
  const int stages = (p.count + GRADIENT_ROWS - 1) / GRADIENT_ROWS;
  unsigned char* to = a.parts[side] + first_stage(p, a.unit) * S::HIDDEN;
  const int stop = min(stages * GRADIENT_ROWS, (int)(blockIdx.z + 1) * SPLIT_ROWS);
  for (int r = blockIdx.z * SPLIT_ROWS + tid / G; r < stop; r += 256 / G) {
    float v[8];
    load(r, v);
    uint4 hi, lo;
    split2<T>(v[0] * s[0], v[1] * s[1], hi.x, lo.x);
    split2<T>(v[2] * s[2], v[3] * s[3], hi.y, lo.y);
    split2<T>(v[4] * s[4], v[5] * s[5], hi.z, lo.z);
    split2<T>(v[6] * s[6], v[7] * s[7], hi.w, lo.w);
    unsigned char* stage = to + (int64_t)(r / GRADIENT_ROWS) * S::HIDDEN;
    const int row = r % GRADIENT_ROWS, ch = lane8, cl = G + lane8;
    *reinterpret_cast<uint4*>(stage + (ch >> 3) * S::PANEL + swizzled(row, ch & 7)) = hi;
    *reinterpret_cast<uint4*>(stage + (cl >> 3) * S::PANEL + swizzled(row, cl & 7)) = lo;
  }
}

template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(TENSOR_THREADS, 2) adapter_gradient_kernel(const OuterArgs a) {
  using S = GradientShared<R>;
  constexpr int ST = S::STAGES;
  constexpr bool SCALED = !std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char raw[];
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  __shared__ Piece found;
  __shared__ uint64_t arrived[ST], freed[ST];  // copies in, products done
  __shared__ uint64_t last;                    // (as in adapter_tensor.cuh)
  __shared__ uint32_t tmem_at;
  __shared__ volatile int gave_up;
  __shared__ int row_of[1024];
  __shared__ float back_of[SCALED ? R : 1];  // the ranks' powers of two
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Piece p;
  if (a.group_of) {  // (as in adapter_tensor.cuh)
    pdl_wait();
    pdl_trigger();
    p = find_piece(a.starts, a.rows, a.groups, a.unit, blockIdx.x, &found);
    if (p.group < 0) return;
  }
  // (set up while the kernels before run)
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&arrived[i], VEC ? ADAPTER_THREADS : 2 * ADAPTER_THREADS);
      mbar_init(&freed[i], 1);
    }
    mbar_init(&last, 1);
    gave_up = 0;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_at, 2 * S::D);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  if (!a.group_of) {
    pdl_wait();
    pdl_trigger();
    p = find_piece(a.starts, a.rows, a.groups, a.unit, blockIdx.x, &found);
  }
  const int side = blockIdx.y < a.blocks[0] ? 0 : 1;  // down's gradient, then up's
  const int adapter = p.group < 0 ? a.L : adapter_of(a, p.group);
  if (adapter == a.L) {  // (rows without one have no factors)
    if (warp == 0) tmem_dealloc(tmem, 2 * S::D);
    return;
  }
  const int n0 = (blockIdx.y - (side ? a.blocks[0] : 0)) * GRADIENT_COLUMNS, N = a.width[side];
  const T* x = static_cast<const T*>(a.x[side]);
  const int64_t stride = a.stride[side];
  for (int r = tid; r < p.count; r += TENSOR_THREADS) row_of[r] = a.row_list[p.start + r];
  if (SCALED && tid < a.rank) back_of[tid] = a.back[side][(int64_t)blockIdx.x * a.rank + tid];
  __syncthreads();
  const Waits wait(&gave_up, a.silent);

  const int stages = (p.count + GRADIENT_ROWS - 1) / GRADIENT_ROWS;
  const unsigned char* parts = a.parts[side] + first_stage(p, a.unit) * S::HIDDEN;
  // a warp copies whole rows: 32 chunks of 16 bytes, four rows a warp
  const int col = n0 + lane * 8;
  const bool in = col < N;
  constexpr int Q = GRADIENT_ROWS / ADAPTER_WARPS;
  const auto issue = [&](int i) {
    const uint32_t at = ring + (i % ST) * S::STAGE;
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int row = warp + q * ADAPTER_WARPS, r = i * GRADIENT_ROWS + row;
        const bool on = in && r < p.count;
        copy16(at + (lane >> 3) * S::PANEL + swizzled(row, lane & 7), on ? x + row_of[r] * stride + col : x, on);
      }
    }
#pragma unroll
    for (int c = tid; c < S::HIDDEN / 16; c += ADAPTER_THREADS)
      copy16(at + S::X + c * 16, parts + (int64_t)i * S::HIDDEN + c * 16, true);
  };
  Loose lx[VEC ? 1 : Q];
  bool odd[VEC ? 1 : Q];
  const auto fetch = [&](int i) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = i * GRADIENT_ROWS + warp + q * ADAPTER_WARPS;
      const bool on = in && r < p.count;
      const T* at = on ? x + row_of[r] * stride + col : x;
      lx[q].load(at, N - col, on);
      odd[q] = Loose::odd(at);
    }
  };
  const auto put = [&](int i) {
    const uint32_t at = ring + (i % ST) * S::STAGE;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      put16(at + (lane >> 3) * S::PANEL + swizzled(warp + q * ADAPTER_WARPS, lane & 7), lx[q].chunk(odd[q], N - col));
  };
  if (warp == ADAPTER_WARPS) {
    if (lane == 0)
      for (int i = 0; i < stages; ++i) {
        if (!wait.alone(i == 0 && a.silent ? &last : &arrived[i % ST], (i / ST) & 1)) break;
        fence_async_shared();
        const uint32_t at = ring + (i % ST) * S::STAGE;
#pragma unroll
        for (int k = 0; k < GRADIENT_ROWS / 16; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < S::PARTS; ++q) {
              // (128 ranks: two panels of first parts, two of second ones)
              const int to = R > 64 ? q & 1 : 0, first = R > 64 ? q < 2 : q == 0;
              tc_mma_f16(tmem + m * S::D + to * 64, smem_desc_rows(at + 2 * m * S::PANEL + k * 2048, S::PANEL),
                         smem_desc_rows(at + S::X + q * S::PANEL + k * 2048), idesc_f16<T>(S::N, true, true),
                         i > 0 || k > 0 || !first);
            }
        tc_commit(&freed[i % ST]);
      }
    __syncwarp();
  } else {
    if constexpr (!VEC) fetch(0);
    for (int i = 0; i < stages; ++i) {
      if (i >= ST && !wait.warp(&freed[i % ST], ((i - ST) / ST) & 1)) break;
      issue(i);
      if constexpr (!VEC) {
        put(i);
        if (i + 1 < stages) fetch(i + 1);
        mbar_arrive(&arrived[i % ST]);  // (for what it has stored itself)
      }
      copy_arrive(&arrived[i % ST]);
    }
  }
  copy_wait_all();
  __syncthreads();
  // (The last commit covers all before.  Whether it was made is known here only: its
  // barrier's phase before would pass for it.)
  const bool ok = __all_sync(0xffffffffu, !gave_up) && wait.warp(&freed[(stages - 1) % ST], ((stages - 1) / ST) & 1);
  tc_fence_after();

  if (warp < ADAPTER_WARPS) {
    // A lane has a column of x, its ranks side by side in tensor memory.
    const int quarter = warp & 3, m = warp >> 2, c = n0 + m * 128 + quarter * 32 + lane;
    const float lost = ok ? 0.0f : NAN;
    const int64_t n = (int64_t)a.rank * N;
    const bool alone = a.starts[p.group + 1] - a.starts[p.group] <= a.unit;  // (the adapter's only piece)
    float* sums = a.sums[side] + (first_sums(p.start - p.number * a.unit, a.unit) + p.number) * n + c;
    T* grad = static_cast<T*>(a.grad[side]) + adapter * n + c;
  #pragma unroll
    for (int r0 = 0; r0 < R; r0 += 8) {
      float v[8] = {}, w[8] = {};
      const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + m * S::D + r0;
      if (ok) {
        tmem_ld8(at, v);
        if (R <= 32) tmem_ld8(at + R, w);  // (the parts have columns of their own)
        tmem_ld_wait();
      }
  #pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r0 + i >= a.rank || c >= N) continue;
        const float f = (R <= 32 ? v[i] + w[i] : v[i]) * (SCALED ? back_of[r0 + i] : 1.0f) + lost;
        if (alone)
          grad[(int64_t)(r0 + i) * N] = from_f32<T>(f);
        else
          sums[(int64_t)(r0 + i) * N] = f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (gave_up) wait.settle(&last, 0, warp == ADAPTER_WARPS && lane == 0);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * S::D);
  }
}

// A factor's gradient: its pieces' sums in order, rounded once; zeros for an
// adapter without rows (of many adapters they are written beforehand).
template <typename T>
__global__ void __launch_bounds__(256) adapter_join_kernel(const OuterArgs a) {
  pdl_wait();
  const int side = blockIdx.z, group = blockIdx.x, adapter = adapter_of(a, group);
  if (adapter < 0 || adapter == a.L) return;
  const int64_t n = (int64_t)a.rank * a.width[side];
  const int lo = a.starts[group], hi = a.starts[group + 1];
  const int parts = (hi - lo + a.unit - 1) / a.unit;
  if (parts == 1) return;  // (written already)
  const float* sums = a.sums[side] + first_sums(lo, a.unit) * n;
  T* out = static_cast<T*>(a.grad[side]) + adapter * n;
  constexpr int U = 4;  // elements and pieces whose loads are in flight together
  for (int64_t i = (int64_t)blockIdx.y * 256 * U + threadIdx.x; i < n; i += (int64_t)gridDim.y * 256 * U) {
    float s[U] = {};
    for (int p = 0; p < parts; p += U) {
      float v[U][U];
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int e = 0; e < U; ++e) v[q][e] = p + q < parts && i + e * 256 < n ? sums[(p + q) * n + i + e * 256] : 0.0f;
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int e = 0; e < U; ++e) s[e] += v[q][e];
    }
#pragma unroll
    for (int e = 0; e < U; ++e)
      if (i + e * 256 < n) out[i + e * 256] = from_f32<T>(s[e]);
  }
}

template <typename T, int R, bool VEC>
cudaError_t launch_gradient_one(const OuterArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = adapter_gradient_kernel<T, R, VEC>;
  cudaError_t e = raise_shared(kernel, GradientShared<R>::BYTES, done);
  if (e != cudaSuccess) return e;
  const unsigned pieces = (unsigned)pieces_of(a.rows, a.groups, a.unit);
  e = launch_k(adapter_split_kernel<T, R>, dim3(pieces, 2, (unsigned)(a.unit / SPLIT_ROWS)), dim3(256), 0, s, true,
               a);
  if (e != cudaSuccess) return e;
  e = launch_k(kernel, dim3(pieces, (unsigned)(a.blocks[0] + a.blocks[1])), dim3(TENSOR_THREADS),
               GradientShared<R>::BYTES, s, true, a);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)a.rank * std::max(a.width[0], a.width[1]);
  // (of many groups few have several pieces: fewer CTAs each)
  const int64_t most = std::max<int64_t>(16384 / a.groups, 4);
  const dim3 grid((unsigned)a.groups, (unsigned)std::min<int64_t>((n + 1023) / 1024, a.group_of ? most : 1024), 2);
  return launch_k(adapter_join_kernel<T>, grid, dim3(256), 0, s, true, a);
}

template <typename T>
cudaError_t launch_gradient(const OuterArgs& a, bool vec, cudaStream_t s) {
  if (a.rank <= 16) return vec ? launch_gradient_one<T, 16, true>(a, s) : launch_gradient_one<T, 16, false>(a, s);
  if (a.rank <= 32) return vec ? launch_gradient_one<T, 32, true>(a, s) : launch_gradient_one<T, 32, false>(a, s);
  if (a.rank <= 64) return vec ? launch_gradient_one<T, 64, true>(a, s) : launch_gradient_one<T, 64, false>(a, s);
  return vec ? launch_gradient_one<T, 128, true>(a, s) : launch_gradient_one<T, 128, false>(a, s);
}

}  // namespace moe
