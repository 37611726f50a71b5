// kernels_adapter.cu - low-rank adapters of many requests: rows grouped by their
// adapter, and the launches of a forward and of the gradients.
#include <algorithm>

#include "adapter_common.cuh"

namespace moe {
namespace {

constexpr int PLAN_THREADS = 1024;
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

// Group blockIdx.x (an adapter, or L for rows without one): its first place,
// the number of rows of the groups before it, and its rows in ascending order.
// Every CTA goes through all ids, 16 a thread and round (up to 16384 rows, once):
// no CTA waits for another.  (16384 rows: 4 us; the kernel behind is set up
// meanwhile.)
__global__ void __launch_bounds__(PLAN_THREADS) adapter_plan_kernel(const int32_t* ids, int rows, int L,
                                                                    int32_t* starts, int32_t* row_list) {
  constexpr int PER = 16, ROUND = PLAN_THREADS * PER;
  __shared__ int less_sum[32], warp_sum[32];
  pdl_trigger();
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    if (base == 0 && tid == 0) starts[group] = at;
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
  if (tid == 0) {
    if (rows == 0) starts[group] = 0;
    if (group == L) starts[L + 1] = rows;
  }
}

int64_t words16(int64_t n) { return (n + 3) / 4 * 4; }

// Where the parts of a workspace lie, in 4-byte words, 16-byte aligned.
struct Layout {
  int64_t starts, row_list, hidden, back, parts[2], sums[2], end;
};

int outer_unit(int64_t rows) {
  // about sixteen pieces of a large batch: with a side's column blocks that fills
  // the SMs, and the pieces' FP32 sums stay small beside the rows
  const int64_t unit = (rows + 15) / 16;
  return (int)std::min<int64_t>(std::max<int64_t>((unit + 63) / 64 * 64, 64), 1024);
}

Layout layout(const moe_adapter_config& c, int64_t rows, bool backward) {
  Layout l{};
  l.starts = 0;
  l.row_list = words16(c.num_adapters + 2);
  l.hidden = l.row_list + words16(rows);
  const int unit = outer_unit(rows);
  const int64_t pieces = backward ? pieces_of(rows, c.num_adapters, unit) : 0;
  // (two 16-bit parts of up to 16, 32, 64 or 128 ranks in rows of 128 bytes)
  const int64_t stages = backward ? pieces_of(rows, c.num_adapters, GRADIENT_ROWS) : 0;
  const int64_t part = stages * GRADIENT_ROWS * (c.rank <= 32 ? 1 : c.rank <= 64 ? 2 : 4) * 32;
  const int64_t sums = backward ? 2 * rows / unit + 1 : 0;
  l.back = l.hidden + (backward ? words16(rows * c.rank) : 0);
  l.parts[0] = l.back + words16(2 * pieces);
  l.parts[1] = l.parts[0] + part;
  l.sums[0] = l.parts[1] + part;
  l.sums[1] = l.sums[0] + words16(sums * c.rank * c.in_features);
  l.end = l.sums[1] + words16(sums * c.rank * c.out_features);
  return l;
}

cudaError_t launch_plan(const AdapterArgs& a, cudaStream_t s) {
  return launch_k(adapter_plan_kernel, dim3((unsigned)a.L + 1), dim3(PLAN_THREADS), 0, s, false, a.ids, (int)a.rows,
                  a.L, const_cast<int32_t*>(a.starts), const_cast<int32_t*>(a.row_list));
}

// CTAs of a cluster: as many as keep the likely tiles within one wave of two
// CTAs an SM (half of the adapters' last tiles count: which are used is known
// on the device only).  16384 rows, rank 64: two 89 us, one 108, four 122; 4096
// rows, rank 16: eight 31, four 39.
int cluster_of(int64_t tiles, int64_t rows, int L) {
  const int64_t full = std::min<int64_t>(rows, (rows + ADAPTER_TILE - 1) / ADAPTER_TILE + std::min<int64_t>(L, rows) / 2);
  const int64_t t = std::max<int64_t>(std::min(tiles, full), 1);
  return t * 8 <= 304 ? 8 : t * 4 <= 304 ? 4 : t * 2 <= 304 ? 2 : 1;
}

cudaError_t apply(AdapterArgs a, bool f16, bool vec, bool planned, cudaStream_t s) {
  a.tiles = planned ? pieces_of(a.rows, a.L + 1, ADAPTER_TILE) : a.L + 1;
  a.cluster = cluster_of(a.tiles, a.rows, a.L);
  if (planned) return f16 ? launch_tensor_f16(a, vec, s) : launch_tensor_bf16(a, vec, s);
  return f16 ? launch_apply_f16(a, vec, s) : launch_apply_bf16(a, vec, s);
}

}  // namespace

size_t adapter_workspace(const moe_adapter_config& c, int64_t rows, bool backward) {
  if (!backward && rows <= ADAPTER_TILE) return 0;
  return (size_t)layout(c, rows, backward).end * 4;
}

cudaError_t launch_adapter(AdapterArgs a, const moe_adapter_config& c, bool vec, void* workspace, cudaStream_t s) {
  const Layout l = layout(c, a.rows, false);
  int32_t* w = static_cast<int32_t*>(workspace);
  a.starts = w + l.starts;
  a.row_list = w + l.row_list;
  const bool planned = a.rows > ADAPTER_TILE;
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
  a.hidden = reinterpret_cast<float*>(w + l.hidden);
  const bool f16 = c.dtype == MOE_DTYPE_F16;
  cudaError_t e = launch_plan(a, s);
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
    o.back[i] = reinterpret_cast<float*>(w + l.back) + i * pieces_of(a.rows, a.L, o.unit);
  }
  return f16 ? launch_gradient_f16(o, vec, s) : launch_gradient_bf16(o, vec, s);
}

}  // namespace moe
