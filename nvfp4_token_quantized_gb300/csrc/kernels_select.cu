// kernels_select.cu - choice of experts from logits (scores, balance bias,
// groups, top-k, renormalised weights) and the gradient of its weights.
#include <atomic>
#include <type_traits>

#include "elem_types.cuh"
#include "kernels_ops.h"
#include "route_select.cuh"
#include "select_parts.cuh"

namespace moe {

namespace {

constexpr int SELECT_WARPS = 8;

__device__ __forceinline__ constexpr int type_of(float) { return MOE_DTYPE_F32; }
__device__ __forceinline__ constexpr int type_of(__half) { return MOE_DTYPE_F16; }
__device__ __forceinline__ constexpr int type_of(__nv_bfloat16) { return MOE_DTYPE_BF16; }

// A warp a row (64 x 256, sigmoid with a bias, 4 of 8 groups, top-8: 3.2 us, of
// which a launch is 2).
template <int NE>
__global__ void __launch_bounds__(32 * SELECT_WARPS)
    select_kernel(const RouteRule r, const void* __restrict__ logits, int dtype, int64_t stride,
                  const float* __restrict__ bias, int64_t rows, int32_t* __restrict__ ids, float* __restrict__ w) {
  __shared__ __align__(16) SelectScratch scratch[SELECT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * SELECT_WARPS + warp;
  pdl_trigger();
  pdl_wait();
  if (t >= rows) return;
  float b[NE];
  const bool finite = load_bias<NE>(r, bias, lane, b);
  select_row<NE>(r, row_at(logits, dtype, t * stride), dtype, bias, b, finite, lane, scratch[warp], ids + t * r.K,
                 w + t * r.K);
}

// Gradient.  A warp takes RB rows at a time, whose slots fit its lanes: first
// the slots, whose values go to their experts' places in shared memory (zero
// elsewhere), then whole rows, so that every element is stored once, four at a
// time where rows allow.  Bytes bound it (131072 x 256 FP32, sigmoid, top-8: 31 us,
// 4.9 TB/s).  Memory answers a scattered logit
// with 64 bytes, so the sigmoid's gradient takes the scores from the weights:
// w = scale s / (sum + 1e-20), and one logit a row (of the largest weight)
// gives the quotient; without renormalisation it needs none.  That leaves
// scores a few 2^-24 off, which 1 - s would magnify where s is near 1: scores
// above NEAR_ONE take both from their logits.  (FP32, 131072 x 256: error against
// 64 bits 1.7 times that of scores from all logits and a difference, at 31 us;
// all logits read: 0.5 times, at 41.)
template <typename T, int NE, int RB, bool SIGMOID>
__global__ void __launch_bounds__(32 * SELECT_WARPS) select_backward_kernel(
    const RouteRule r, const T* logits, int64_t stride, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, int64_t rows, T* dlogits, int64_t dstride) {
  constexpr int WIDTH = NE * 32;
  // (1 - s keeps 16 bits or more of the FP32 ones, 14 for the 16-bit types,
  // whose results have 11)
  constexpr float NEAR_ONE = sizeof(T) == 4 ? 1.0f - 1.0f / 64 : 1.0f - 1.0f / 256;
  __shared__ __align__(16) float place[SELECT_WARPS][RB][WIDTH];
  const unsigned all = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float(*buf)[WIDTH] = place[warp];
  for (int i = lane; i < RB * WIDTH; i += 32) buf[0][i] = 0.0f;
  __syncwarp();
  const int slots = 1 << r.slot_shift;
  const int my_q = lane >> r.slot_shift, c = lane & (slots - 1);
  const int64_t step = (int64_t)gridDim.x * SELECT_WARPS * RB;
  auto over_slots = [&](float x) {
#pragma unroll 1
    for (int o = slots >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(all, x, o);
    return x;
  };
  for (int64_t t = ((int64_t)blockIdx.x * SELECT_WARPS + warp) * RB; t < rows; t += step) {
    const int valid = rows - t < RB ? (int)(rows - t) : RB;
    // this lane's slot; id -1: no gradient
    int id = -1;
    float weight = 0.0f, d = 0.0f;
    if (my_q < valid && c < r.K) {
      const int64_t at = (t + my_q) * r.K + c;
      weight = __ldg(w + at);
      d = __ldg(dw + at) * r.scale;
      id = __ldg(ids + at);
    }
    float p[RB][NE];  // softmax: the rows' scores
    if constexpr (!SIGMOID) {
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        if (q < valid) {
          load_logits<NE>(r, logits + (t + q) * stride, type_of(T()), lane, p[q]);
        } else {
#pragma unroll
          for (int i = 0; i < NE; ++i) p[q][i] = -INFINITY;
        }
      }
    }
    if (weight == 0.0f || (unsigned)id >= (unsigned)r.E) id = -1;
    if (id < 0) d = 0.0f;
    float score = 0.0f, sum = 1.0f;  // sum: of the chosen scores, plus 1e-20
    float rest = 1.0f;               // 1 - score (sigmoid)
    if constexpr (SIGMOID) {
      score = id >= 0 ? weight / r.scale : 0.0f;
      if (r.renormalize) {
        // (score so far: s / sum)
        float most = fabsf(score);
#pragma unroll 1
        for (int o = slots >> 1; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(all, most, o));
        const unsigned top = __ballot_sync(all, id >= 0 && fabsf(score) == most) >> (my_q << r.slot_shift);
        const int leader = (my_q << r.slot_shift) + (top ? __ffs(top) - 1 : 0);
        float whole = __int_as_float(0x7fffffff);
        if (lane == leader && id >= 0) whole = sigmoid_ieee(to_f32(logits[(t + my_q) * stride + id])) / score;
        sum = __shfl_sync(all, whole, leader);
        score = id >= 0 ? score * sum : 0.0f;
      }
      rest = 1.0f - score;
      if (id >= 0 && !(score < NEAR_ONE)) {
        const float e = expf(-to_f32(logits[(t + my_q) * stride + id]));
        score = 1.0f / (1.0f + e);
        rest = e * score;
      }
    } else {
      float my_top = 0.0f, my_total = 1.0f;
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        float m = p[q][0];
#pragma unroll
        for (int i = 1; i < NE; ++i) m = fmaxf(m, p[q][i]);
        m = max_lanes(m);
        if (m == -INFINITY) m = 0.0f;
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          p[q][i] = expf(p[q][i] - m);
          total += p[q][i];
        }
        total = sum_lanes(total);
        if (total == 0.0f) total = 1.0f;
        const float k = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NE; ++i) p[q][i] *= k;
        if (my_q == q) my_top = m, my_total = total;
      }
      if (id >= 0) score = expf(to_f32(logits[(t + my_q) * stride + id]) - my_top) / my_total;
      if (r.renormalize) sum = over_slots(score) + SELECT_SUM_EPS;
    }
    if (r.renormalize) {
      const float along = over_slots(d * score) / sum;
      d = id >= 0 ? (d - along) / sum : 0.0f;
    }
    float my_mean = 0.0f;  // of the row of this lane's slot
    if constexpr (SIGMOID) d *= score * rest;
    else my_mean = over_slots(d * score);
    if (id >= 0) buf[my_q][id] = d;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const float mean = SIGMOID ? 0.0f : __shfl_sync(all, my_mean, q << r.slot_shift);
      if (q >= valid) break;
      T* out = dlogits + (t + q) * dstride;
      if (r.vec) {
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
          const int e = (i / 4 * 32 + lane) * 4;
          if (e >= r.E) break;
          float4 f = *reinterpret_cast<const float4*>(&buf[q][e]);
          if constexpr (!SIGMOID)
            f = make_float4(p[q][i] * (f.x - mean), p[q][i + 1] * (f.y - mean), p[q][i + 2] * (f.z - mean),
                            p[q][i + 3] * (f.w - mean));
          if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(out + e) = f;
          else *reinterpret_cast<uint2*>(out + e) = make_uint2(pack2(f.x, f.y, T()), pack2(f.z, f.w, T()));
        }
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int e = i * 32 + lane;
          if (e >= r.E) break;
          const float f = buf[q][e];
          out[e] = from_f32<T>(SIGMOID ? f : p[q][i] * (f - mean));
        }
      }
    }
    __syncwarp();
    if (id >= 0) buf[my_q][id] = 0.0f;
    __syncwarp();
  }
}

template <int NE>
cudaError_t launch_select_rows(const RouteRule& r, const void* logits, int dtype, int64_t stride, const float* bias,
                               int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s) {
  return launch_k(select_kernel<NE>, dim3((unsigned)((rows + SELECT_WARPS - 1) / SELECT_WARPS)),
                  dim3(32 * SELECT_WARPS), 0, s, pdl, r, logits, dtype, stride, bias, rows, ids, w);
}

// More parts a row leave more warps, whose loads hide one another's latency,
// and fewer columns a thread: 65536 x 128 takes 17.4 us with four of 32, 23.9
// with two of 64 and 36.4 with one of 128; 131072 x 256 in eight groups 69, 71
// (eight of 32) and 87 (two of 128).
template <int R, int P>
cudaError_t launch_select_parts(const RouteRule& r, const void* logits, int dtype, int64_t stride, const float* bias,
                                int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s) {
  using L = PartLayout<R, P>;
  return launch_k(select_parts_kernel<R, P>, dim3((unsigned)((rows + L::ROWS - 1) / L::ROWS)), dim3(32),
                  L::words(r) * sizeof(float), s, pdl, r, logits, dtype, stride, bias, rows, ids, w);
}

template <typename T, int NE, int RB, bool SIGMOID>
cudaError_t launch_backward_rows(const RouteRule& r, const T* logits, int64_t stride, const int32_t* ids,
                                 const float* w, const float* dw, int64_t rows, T* dlogits, int64_t dstride,
                                 cudaStream_t s) {
  auto kernel = select_backward_kernel<T, NE, RB, SIGMOID>;
  static std::atomic<int> resident{0};  // CTAs an SM holds; 0: not asked yet
  int ctas = resident.load(std::memory_order_relaxed);
  if (ctas == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, 32 * SELECT_WARPS, 0);
    if (e != cudaSuccess) return e;
    ctas = ctas > 0 ? ctas : 1;
    resident.store(ctas, std::memory_order_relaxed);
  }
  // one wave; its warps walk the rows
  const int64_t need = (rows + SELECT_WARPS * RB - 1) / (SELECT_WARPS * RB);
  return launch_k(kernel, dim3((unsigned)(need < 152 * ctas ? need : 152 * ctas)), dim3(32 * SELECT_WARPS), 0, s,
                  false, r, logits, stride, ids, w, dw, rows, dlogits, dstride);
}

template <typename T>
cudaError_t select_backward_t(RouteRule r, const void* logits, int64_t stride, const int32_t* ids, const float* w,
                              const float* dw, int64_t rows, void* dlogits, int64_t dstride, cudaStream_t s) {
  // the choice is given: one group
  r.groups = r.top_groups = 1;
  r.size = r.E;
  r.lane_shift = 5;
  const T* l = static_cast<const T*>(logits);
  T* d = static_cast<T*>(dlogits);
  const uintptr_t at = reinterpret_cast<uintptr_t>(l) | reinterpret_cast<uintptr_t>(d);
  r.vec = r.E % 4 == 0 && (stride | dstride) % 4 == 0 && (at & (4 * sizeof(T) - 1)) == 0;
  auto go = [&](auto width, auto batch) {
    constexpr int NE = decltype(width)::value, RB = decltype(batch)::value;
    if (r.sigmoid) return launch_backward_rows<T, NE, RB, true>(r, l, stride, ids, w, dw, rows, d, dstride, s);
    return launch_backward_rows<T, NE, RB, false>(r, l, stride, ids, w, dw, rows, d, dstride, s);
  };
  // rows a warp takes at a time: as many as have room for their slots, up to
  // four, once that keeps every scheduler busy
  using std::integral_constant;
  auto width = [&](auto batch) {
    if (r.E <= 128) return go(integral_constant<int, 4>{}, batch);
    if constexpr (decltype(batch)::value == 4) {
      return go(integral_constant<int, 8>{}, batch);
    } else {
      if (r.E <= 256) return go(integral_constant<int, 8>{}, batch);
      return go(integral_constant<int, 16>{}, batch);
    }
  };
  if (rows < 152 * 4 * 4 * 4 || r.slot_shift > 4) return width(integral_constant<int, 1>{});
  if (r.slot_shift > 3 || r.E > 256) return width(integral_constant<int, 2>{});
  return width(integral_constant<int, 4>{});
}

}  // namespace

cudaError_t launch_select(const RouteRule& rule, const void* logits, int dtype, int64_t stride, const float* bias,
                          int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s) {
  RouteRule r = rule;
  const int bytes = dtype == MOE_DTYPE_F32 ? 4 : 2;
  const bool aligned = stride % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & (4 * bytes - 1)) == 0;
  // Parts of rows once they make five warps an SM, which is where the two
  // meet (128 experts, all open: 4096 rows 5.2 us against a warp a row's 4.6,
  // 8192 rows 6.1 against 7.5, 16384 7.5 against 12.3).
  const int parts = r.E <= 64 ? 2 : 4;
  if (rows * parts >= 32 * 5 * 152) {
    r.vec = aligned && r.E % 4 == 0;
    if (r.E <= 64) return launch_select_parts<1, 2>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
    if (r.E <= 128) return launch_select_parts<1, 4>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
    if (r.E <= 256) return launch_select_parts<2, 4>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
    return launch_select_parts<4, 4>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  }
  set_select_loads(r, aligned);
  const int n = select_per_lane(r);
  if (n <= 4) return launch_select_rows<4>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  if (n <= 8) return launch_select_rows<8>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  if (n <= 16) return launch_select_rows<16>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
  return launch_select_rows<32>(r, logits, dtype, stride, bias, rows, ids, w, pdl, s);
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
