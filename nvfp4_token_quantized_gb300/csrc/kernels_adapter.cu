// kernels_adapter.cu - low-rank adapters of many requests: rows grouped by their
// adapter, and the launches of a forward and of the gradients.
#include <algorithm>
#include <type_traits>

#include "adapter_common.cuh"

namespace moe {
namespace {

constexpr int PLAN_THREADS = 1024, PLAN_CTAS = 304;  // (two an SM)
constexpr unsigned ALL = 0xffffffffu;

// Sixteen neighbouring ids, as groups (-1 from `rows` on).
__device__ __forceinline__ void load_groups(const int32_t* ids, int64_t first, int rows, int L, int (&g)[16]) {
  if (first + 16 <= rows && ((uintptr_t)(ids + first) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int4 v = reinterpret_cast<const int4*>(ids + first)[i];
      g[4 * i] = v.x, g[4 * i + 1] = v.y, g[4 * i + 2] = v.z, g[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = adapter_key(g[i], L);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = first + i < rows ? adapter_key(ids[first + i], L) : -1;
  }
}

constexpr int MAX_WORDS = (65536 + 32) / 32 + 1;  // a bit for each adapter and for none

// The adapters with rows (L: rows without one), numbered in ascending order: all
// threads mark the adapters they meet, then count.
struct Present {
  static constexpr int EACH = (MAX_WORDS + PLAN_THREADS - 1) / PLAN_THREADS;
  unsigned marks[EACH * PLAN_THREADS];
  int sums[32], result;
  // Returns the number of those before this thread's words, and of all.
  __device__ __forceinline__ int2 mark(const int32_t* ids, int rows, int L) {
    constexpr int PER = 16, ROUND = PLAN_THREADS * PER;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < EACH * PLAN_THREADS; i += PLAN_THREADS) marks[i] = 0;
    __syncthreads();
    for (int64_t base = 0; base < rows; base += ROUND) {
      int g[PER];
      load_groups(ids, base + tid * PER, rows, L, g);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (g[i] >= 0 && !(*(volatile unsigned*)&marks[g[i] >> 5] >> (g[i] & 31) & 1)) atomicOr(&marks[g[i] >> 5], 1u << (g[i] & 31));
    }
    __syncthreads();
    int mine = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) mine += __popc(marks[tid * EACH + i]);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(ALL, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    const int w = sums[lane];
    return make_int2(__reduce_add_sync(ALL, lane < warp ? w : 0) + upto - mine, __reduce_add_sync(ALL, w));
  }
  // The one of a number that there is.
  __device__ __forceinline__ int pick(int before, int number) {
    const int tid = threadIdx.x;
    for (int i = 0; i < EACH; ++i)
      for (unsigned m = marks[tid * EACH + i]; m; m &= m - 1)
        if (before++ == number) result = (tid * EACH + i) * 32 + __ffs(m) - 1;
    __syncthreads();
    return result;  // (another is written behind the next barrier only)
  }
};

// A group's first place, the number of rows of the groups before it, and its rows in
// ascending order.  Every CTA goes through all ids, 16 a thread and round (up to
// 16384 rows, once): no CTA waits for another.  (16384 rows: 4 us; the kernel behind
// is set up meanwhile.)  COMPACT: only groups with rows, a CTA every so many (4096
// rows of 64 adapters in a set of 4000: the forward in 54 us, with a CTA a group 91).
// The work is rows times groups with rows, which shows from some hundred of those on:
// 16384 rows of 64 present adapters 13 us, of 4000 121; 65536 of 4000 382; 100000 of
// 60000 6.5 ms.  (A sort by counting would be linear in the rows.)
template <bool COMPACT>
__global__ void __launch_bounds__(PLAN_THREADS, 2) adapter_plan_kernel(const int32_t* ids, int rows, int L, int groups,
                                                                    int32_t* starts, int32_t* row_list,
                                                                    int32_t* group_of) {
  constexpr int PER = 16, ROUND = PLAN_THREADS * PER;
  __shared__ int less_sum[32], warp_sum[32];
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0 && blockIdx.x == 0) starts[groups] = rows;
  int2 present = make_int2(0, groups);
  __shared__ std::conditional_t<COMPACT, Present, int> of;
  if constexpr (COMPACT) present = of.mark(ids, rows, L);
  for (int number = blockIdx.x; number < groups; number += gridDim.x) {
    const bool none = rows == 0 || (COMPACT && number >= present.y);
    int group = none ? -1 : number;
    if constexpr (COMPACT) {
      if (!none) group = of.pick(present.x, number);
      if (tid == 0) group_of[number] = group;
    }
    if (none) {
      if (tid == 0) starts[number] = rows;
      continue;
    }
    int g[PER], less = 0;
    for (int64_t base = 0; base < rows; base += ROUND) {
      load_groups(ids, base + tid * PER, rows, L, g);
#pragma unroll
      for (int i = 0; i < PER; ++i) less += (unsigned)g[i] < (unsigned)group;
    }
    less = __reduce_add_sync(ALL, less);
    if (lane == 0) less_sum[warp] = less;
    int at = 0;
    for (int64_t base = 0; base < rows; base += ROUND) {
      if (rows > ROUND) load_groups(ids, base + tid * PER, rows, L, g);  // (else they are still here)
      unsigned mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) mine |= (unsigned)(g[i] == group) << i;
      const int n = __popc(mine);
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(ALL, upto, o);
        if (lane >= o) upto += v;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      if (base == 0) at = __reduce_add_sync(ALL, less_sum[lane]);
      if (base == 0 && tid == 0) starts[number] = at;
      const int w = warp_sum[lane];
      const int before = __reduce_add_sync(ALL, lane < warp ? w : 0), all = __reduce_add_sync(ALL, w);
      int put = at + before + upto - n;
      const int32_t first = (int32_t)(base + tid * PER);
      while (mine) {
        row_list[put++] = first + __ffs(mine) - 1;
        mine &= mine - 1;
      }
      at += all;
      __syncthreads();  // (the next round overwrites the warps' sums)
    }
    if constexpr (!COMPACT) return;  // (a CTA a group)
  }
}

int64_t words16(int64_t n) { return (n + 3) / 4 * 4; }

// Where the parts of a workspace lie, in 4-byte words, 16-byte aligned.
struct Layout {
  int64_t starts, row_list, group_of, hidden, back, parts[2], sums[2], end;
};

// Groups of a call.  Of few adapters each is one, with rows or without; of more only
// as many as rows can have: a tile's number each, for a search of 4 us (300 rows,
// planned: 64 adapters 32 and 36 us, 256 52 and 55, 1000 91 and 51).
constexpr int FEW_GROUPS = 256;
bool few_groups(int L) { return L < FEW_GROUPS; }
int groups_of(int64_t rows, int L) { return (int)(few_groups(L) ? L + 1 : std::min<int64_t>(L + 1, std::max<int64_t>(rows, 1))); }

int outer_unit(int64_t rows) {
  // about sixteen pieces of a large batch: with a side's column blocks that fills
  // the SMs, and the pieces' FP32 sums stay small beside the rows
  const int64_t unit = (rows + 15) / 16;
  return (int)std::min<int64_t>(std::max<int64_t>((unit + 63) / 64 * 64, 64), 1024);
}

Layout layout(const moe_adapter_config& c, int64_t rows, bool backward) {
  Layout l{};
  l.starts = 0;
  const int groups = groups_of(rows, c.num_adapters);
  l.row_list = words16(groups + 1);
  l.group_of = l.row_list + words16(rows);
  l.hidden = l.group_of + words16(groups);
  const int unit = outer_unit(rows);
  const int64_t pieces = backward ? pieces_of(rows, groups, unit) : 0;
  // (two 16-bit parts of up to 16, 32, 64 or 128 ranks in rows of 128 bytes)
  const int64_t stages = backward ? pieces_of(rows, groups, GRADIENT_ROWS) : 0;
  const int64_t part = stages * GRADIENT_ROWS * (c.rank <= 32 ? 1 : c.rank <= 64 ? 2 : 4) * 32;
  const int64_t sums = backward ? 2 * rows / unit + 1 : 0;
  l.back = l.hidden + (backward ? words16(rows * c.rank) : 0);
  l.parts[0] = l.back + words16(2 * pieces * c.rank);
  l.parts[1] = l.parts[0] + part;
  l.sums[0] = l.parts[1] + part;
  l.sums[1] = l.sums[0] + words16(sums * c.rank * c.in_features);
  l.end = l.sums[1] + words16(sums * c.rank * c.out_features);
  return l;
}

cudaError_t launch_plan(const AdapterArgs& a, cudaStream_t s) {
  const bool compact = a.group_of != nullptr;
  const unsigned grid = (unsigned)(compact ? std::min(a.groups, PLAN_CTAS) : a.groups);
  return launch_k(compact ? adapter_plan_kernel<true> : adapter_plan_kernel<false>, dim3(grid), dim3(PLAN_THREADS), 0, s,
                  false, a.ids, (int)a.rows, a.L, a.groups, const_cast<int32_t*>(a.starts),
                  const_cast<int32_t*>(a.row_list), const_cast<int32_t*>(a.group_of));
}

// CTAs of a cluster: as many as keep the likely tiles within one wave of two
// CTAs an SM.  Which adapters have rows is known on the device only: half of
// their last tiles count, and a quarter for the step from one CTA to two (a CTA
// alone takes all of both long axes).  16384 rows, rank 64: two 89 us, one 108,
// four 122; 4096 rows, rank 16: eight 31, four 39; 2048 rows, rank 16, of 1, 8,
// 64 and all of 300 adapters: two 42, 42, 38 and 61 us, one 63, 63, 50 and 54.
int cluster_of(int64_t tiles, int64_t rows, int L) {
  const auto likely = [&](int share) {
    const int64_t full = (rows + ADAPTER_TILE - 1) / ADAPTER_TILE + std::min<int64_t>(L, rows) / share;
    return std::max<int64_t>(std::min(tiles, std::min(rows, full)), 1);
  };
  return likely(2) * 8 <= 304 ? 8 : likely(2) * 4 <= 304 ? 4 : likely(4) * 2 <= 304 ? 2 : 1;
}

// Whether a forward is one launch without a plan.  Above 256 rows the tensor cores'
// path is the faster one where few adapters of higher ranks share the rows.  (160
// rows of 1, 8, 64 and 160 adapters in a set of 300, rank 16, 2048 wide: 16, 16, 14
// and 20 us, planned 35, 33, 35 and 39; 512 rows of 1, 8, 64 and 512: 20, 20, 20 and
// 34, planned 36, 36, 34 and 63.  512 rows, rank 64, 4096 wide, of 8 adapters in a
// set of 8 37 and 28, in one of 64 36 and 34, of all 64 36 and 52.)
bool few_rows(const moe_adapter_config& c, int64_t rows) {
  return rows <= FEW_ROWS / 2 || (rows <= FEW_ROWS && (c.rank <= 32 || c.num_adapters > 32));
}

cudaError_t apply(AdapterArgs a, bool f16, bool vec, bool planned, cudaStream_t s) {
  if (planned) {
    a.tiles = pieces_of(a.rows, a.groups, ADAPTER_TILE);
    a.cluster = cluster_of(a.tiles, a.rows, a.L);
    return f16 ? launch_tensor_f16(a, vec, s) : launch_tensor_bf16(a, vec, s);
  }
  a.subs = (int)((a.rows + APPLY_TILE - 1) / APPLY_TILE);
  a.tiles = std::min<int64_t>((a.L + 1) * (int64_t)a.subs, a.rows);
  // (of more rows four, whoever has them: 300 rows, rank 64, of one adapter, 4096
  // wide, four 29 us, two 44, eight 27; of 300 adapters, 2048 wide, 43, 45 and 56)
  a.cluster = a.rows <= ADAPTER_TILE ? cluster_of(a.tiles, a.rows, a.L) : 4;
  return f16 ? launch_apply_f16(a, vec, s) : launch_apply_bf16(a, vec, s);
}

}  // namespace

size_t adapter_workspace(const moe_adapter_config& c, int64_t rows, bool backward) {
  if (!backward && few_rows(c, rows)) return 0;
  return (size_t)layout(c, rows, backward).end * 4;
}

cudaError_t launch_adapter(AdapterArgs a, const moe_adapter_config& c, bool vec, void* workspace, cudaStream_t s) {
  const Layout l = layout(c, a.rows, false);
  int32_t* w = static_cast<int32_t*>(workspace);
  a.starts = w + l.starts;
  a.row_list = w + l.row_list;
  a.groups = groups_of(a.rows, a.L);
  a.group_of = few_groups(a.L) ? nullptr : w + l.group_of;
  const bool planned = !few_rows(c, a.rows);
  if (planned) {
    const cudaError_t e = launch_plan(a, s);
    if (e != cudaSuccess) return e;
  }
  return apply(a, c.dtype == MOE_DTYPE_F16, vec, planned, s);
}

cudaError_t launch_adapter_backward(AdapterArgs a, OuterArgs o, const moe_adapter_config& c, bool vec, void* workspace,
                                    cudaStream_t s) {
  const Layout l = layout(c, a.rows, true);
  int32_t* w = static_cast<int32_t*>(workspace);
  a.starts = o.starts = w + l.starts;
  a.row_list = o.row_list = w + l.row_list;
  a.groups = o.groups = groups_of(a.rows, a.L);
  a.group_of = o.group_of = few_groups(a.L) ? nullptr : w + l.group_of;
  a.hidden = reinterpret_cast<float*>(w + l.hidden);
  const bool f16 = c.dtype == MOE_DTYPE_F16;
  cudaError_t e = cudaSuccess;
  if (a.group_of)  // (most adapters have no rows, and no group that would write zeros)
    for (int i = 0; i < 2 && e == cudaSuccess; ++i)
      e = cudaMemsetAsync(o.grad[i], 0, (size_t)a.L * a.rank * o.width[i] * 2, s);
  if (e == cudaSuccess) e = launch_plan(a, s);
  if (e == cudaSuccess) e = apply(a, f16, vec, true, s);
  if (e != cudaSuccess) return e;
  o.hidden[0] = a.hidden;  // down's gradient goes by dout up^T, up's by the forward's hidden
  o.sums[0] = reinterpret_cast<float*>(w + l.sums[0]);
  o.sums[1] = reinterpret_cast<float*>(w + l.sums[1]);
  o.rows = a.rows;
  o.L = a.L;
  o.rank = a.rank;
  o.unit = outer_unit(a.rows);
  for (int i = 0; i < 2; ++i) {
    o.blocks[i] = (o.width[i] + 255) / 256;
    o.parts[i] = reinterpret_cast<unsigned char*>(w + l.parts[i]);
    o.back[i] = reinterpret_cast<float*>(w + l.back) + i * pieces_of(a.rows, o.groups, o.unit) * a.rank;
  }
  return f16 ? launch_gradient_f16(o, vec, s) : launch_gradient_bf16(o, vec, s);
}

}  // namespace moe
