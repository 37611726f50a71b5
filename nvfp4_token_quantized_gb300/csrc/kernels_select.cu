// kernels_select.cu - choice of experts from logits (scores, balance bias,
// groups, top-k, renormalised weights) and the gradient of its weights.
#include "elem_types.cuh"
#include "kernels_ops.h"
#include "route_select.cuh"

namespace moe {

namespace {

constexpr int SELECT_WARPS = 8;

// RB rows a warp.
template <int NE, int RB, int MODE>
__global__ void __launch_bounds__(32 * SELECT_WARPS, NE <= 8 ? 3 : 1)
    select_kernel(const RouteRule r, const void* __restrict__ logits, int dtype, int64_t stride,
                  const float* __restrict__ bias, int64_t rows, int32_t* __restrict__ ids, float* __restrict__ w) {
  __shared__ __align__(16) SelectScratch<RB> scratch[SELECT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = ((int64_t)blockIdx.x * SELECT_WARPS + warp) * RB;
  pdl_trigger();
  pdl_wait();
  if (t >= rows) return;
  float b[NE];
  const bool finite = load_bias<NE>(r, bias, lane, b);
  select_rows<NE, RB, MODE>(r, row_at(logits, dtype, t * stride), dtype, stride, (int)(rows - t < RB ? rows - t : RB),
                            bias, b, finite, lane, scratch[warp], ids + t * r.K, w + t * r.K);
}

// One warp per token; lane j < K holds slot j.  Every element gets its part
// that comes from no slot of its own, then the chosen ones are overwritten.
template <typename T>
__global__ void __launch_bounds__(32 * SELECT_WARPS) select_backward_kernel(
    const RouteRule r, const T* logits, int64_t stride, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, int64_t rows, T* dlogits, int64_t dstride) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * SELECT_WARPS + (threadIdx.x >> 5);
  if (t >= rows) return;
  const T* row = logits + t * stride;
  T* drow = dlogits + t * dstride;
  int id = -1;
  float wk = 0.0f, dk = 0.0f;
  if (lane < r.K) {
    id = ids[t * r.K + lane];
    wk = w[t * r.K + lane];
    dk = dw[t * r.K + lane] * r.scale;
    if ((unsigned)id >= (unsigned)r.E) id = -1;
  }
  const bool live = id >= 0 && wk != 0.0f;
  float m = -INFINITY, total = 0.0f;
  if (!r.sigmoid) {
    for (int e = lane; e < r.E; e += 32) m = fmaxf(m, to_f32(row[e]));
    m = max_lanes(m);
    if (m == -INFINITY) m = 0.0f;
    for (int e = lane; e < r.E; e += 32) total += expf(to_f32(row[e]) - m);
    total = sum_lanes(total);
    if (total == 0.0f) total = 1.0f;
  }
  const float l = id >= 0 ? to_f32(row[id]) : 0.0f;
  const float score = id < 0 ? 0.0f : r.sigmoid ? sigmoid_ieee(l) : expf(l - m) / total;
  const float s = live ? score : 0.0f;
  // ds: gradient of this slot's score
  float ds = live ? dk : 0.0f;
  if (r.renormalize) {
    const float sum = sum_lanes(s) + SELECT_SUM_EPS;
    const float along = sum_lanes(ds * s) / sum;
    ds = live ? (dk - along) / sum : 0.0f;
  }
  if (r.sigmoid) {
    __syncwarp();
    for (int e = lane; e < r.E; e += 32) drow[e] = from_f32<T>(0.0f);
    __syncwarp();
    if (live) drow[id] = from_f32<T>(ds * score * (1.0f - score));
    return;
  }
  const float mean = sum_lanes(ds * s);
  __syncwarp();
  for (int e = lane; e < r.E; e += 32) {
    const float p = expf(to_f32(row[e]) - m) / total;
    drow[e] = from_f32<T>(-p * mean);
  }
  __syncwarp();
  if (live) drow[id] = from_f32<T>(score * (ds - mean));
}

template <int NE, int RB, int MODE>
cudaError_t launch_select_rows(const RouteRule& r, const void* logits, int dtype, int64_t stride, const float* bias,
                               int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s) {
  const int64_t per_cta = SELECT_WARPS * RB;
  return launch_k(select_kernel<NE, RB, MODE>, dim3((unsigned)((rows + per_cta - 1) / per_cta)),
                  dim3(32 * SELECT_WARPS), 0, s, pdl, r, logits, dtype, stride, bias, rows, ids, w);
}

// Rows a warp takes together: four (two of up to 16 experts a lane) once that
// still leaves every scheduler a few warps, by kernels compiled for the kind of
// rule; one below, where latency counts, by one kernel for all.
template <int NE, int RB>
cudaError_t select_n(const RouteRule& r, const void* logits, int dtype, int64_t stride, const float* bias,
                     int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s) {
  if (RB == 1 || rows < 152 * 4 * 4 * RB)
    return launch_select_rows<NE, 1, SELECT_ANY>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  if constexpr (RB > 1) {
    const int mode = (r.sigmoid ? SELECT_SIGMOID : 0) | (r.by_score ? SELECT_BY_SCORE : 0) |
                     (r.top_groups < r.groups ? SELECT_LIMITED : 0);
#define MOE_SELECT_MODE(M) \
  case M: return launch_select_rows<NE, RB, M>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s)
    switch (mode) {
      MOE_SELECT_MODE(0);
      MOE_SELECT_MODE(1);
      MOE_SELECT_MODE(2);
      MOE_SELECT_MODE(3);
      MOE_SELECT_MODE(4);
      MOE_SELECT_MODE(5);
      MOE_SELECT_MODE(6);
      MOE_SELECT_MODE(7);
    }
#undef MOE_SELECT_MODE
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t select_backward_t(const RouteRule& r, const void* logits, int64_t stride, const int32_t* ids,
                              const float* w, const float* dw, int64_t rows, void* dlogits, int64_t dstride,
                              cudaStream_t s) {
  const dim3 grid((unsigned)((rows + SELECT_WARPS - 1) / SELECT_WARPS)), block(32 * SELECT_WARPS);
  return launch_k(select_backward_kernel<T>, grid, block, 0, s, false, r, static_cast<const T*>(logits), stride, ids,
                  w, dw, rows, static_cast<T*>(dlogits), dstride);
}

}  // namespace

cudaError_t launch_select(const RouteRule& rule, const void* logits, int dtype, int64_t stride, const float* bias,
                          int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s) {
  RouteRule r = rule;
  const int bytes = dtype == MOE_DTYPE_F32 ? 4 : 2;
  set_select_loads(r, stride % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & (4 * bytes - 1)) == 0);
  const int n = select_per_lane(r);
  if (n <= 4) return select_n<4, 4>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  if (n <= 8) return select_n<8, 4>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  if (n <= 16) return select_n<16, 2>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  return select_n<32, 1>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
}

cudaError_t launch_select_backward(const RouteRule& r, const void* logits, int dtype, int64_t stride,
                                   const int32_t* ids, const float* w, const float* dw, int64_t rows, void* dlogits,
                                   int64_t dstride, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F32)
    return select_backward_t<float>(r, logits, stride, ids, w, dw, rows, dlogits, dstride, s);
  if (dtype == MOE_DTYPE_F16)
    return select_backward_t<__half>(r, logits, stride, ids, w, dw, rows, dlogits, dstride, s);
  return select_backward_t<__nv_bfloat16>(r, logits, stride, ids, w, dw, rows, dlogits, dstride, s);
}

}  // namespace moe
