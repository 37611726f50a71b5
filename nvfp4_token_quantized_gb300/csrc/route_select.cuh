// route_select.cuh - the choice of experts of one token by one warp: scores,
// balance bias, groups, top-k, renormalised weights.  Used by the standalone
// kernel (kernels_select.cu) and the small-batch front kernel
// (kernels_route.cu).
#pragma once

#include "common.cuh"
#include "kernels_ops.h"

namespace moe {

// Bits of a float as an unsigned integer of the same order (-0 as +0).
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float max_lanes(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float sigmoid_ieee(float l) { return 1.0f / (1.0f + expf(-l)); }

// The expert of local slot i of this lane, or -1.
__device__ __forceinline__ int select_expert(const RouteRule& r, int lane, int i) {
  const int lanes = 1 << r.lane_shift;
  const int g = lane >> r.lane_shift, l = lane & (lanes - 1);
  const int o = ((i >> 2) * lanes + l) * 4 + (i & 3);
  return g < r.groups && o < r.size ? g * r.size + o : -1;
}

// raw[i]: the logit of this lane's expert i (-inf where it has none).
// logit(e) reads one logit again, bias(e) the balance bias (0 without one).
// Lane j < K returns slot j in e_lane and w_lane.  All 32 lanes call it.
template <int NE, typename Logit, typename Bias>
__device__ __forceinline__ void select_warp(const RouteRule& r, int lane, const float (&raw)[NE], Logit&& logit,
                                            Bias&& bias, int& e_lane, float& w_lane) {
  float m = -INFINITY, total = 1.0f;
  bool undefined = false;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    undefined |= raw[i] != raw[i] || (!r.sigmoid && raw[i] == INFINITY);
    m = fmaxf(m, raw[i]);
  }
  if (__any_sync(0xffffffffu, undefined)) {
    e_lane = lane;
    w_lane = __int_as_float(0x7fffffff);
    return;
  }
  if (!r.sigmoid) {
    m = max_lanes(m);
    if (m == -INFINITY) m = 0.0f;  // nothing open: every score is 0
    // The sum cancels from renormalised weights (the best logit is among the
    // chosen, so their sum is far above the 1e-20).
    if (r.by_score || !r.renormalize) {
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) total += expf(raw[i] - m);
      total = sum_lanes(total);
      if (total == 0.0f) total = 1.0f;
    }
  }
  // what the choice compares; -inf: closed
  float v[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    v[i] = raw[i];
    if (r.by_score && raw[i] != -INFINITY) {
      const float s = r.sigmoid ? sigmoid_ieee(raw[i]) : expf(raw[i] - m) / total;
      v[i] = s + bias(select_expert(r, lane, i));
      if (!(v[i] > -INFINITY)) v[i] = -INFINITY;  // (NaN too)
    }
  }
  if (r.top_groups < r.groups) {
    const int lanes = 1 << r.lane_shift, g = lane >> r.lane_shift;
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      b2 = fmaxf(b2, fminf(b1, v[i]));
      b1 = fmaxf(b1, v[i]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
      b1 = fmaxf(b1, c1);
    }
    const float gs = r.top2 && b2 > -INFINITY ? b1 + b2 : b1;
    int rank = 0;
    for (int j = 0; j < r.groups; ++j) {
      const float other = __shfl_sync(0xffffffffu, gs, j << r.lane_shift);
      rank += other > gs || (other == gs && j < g);
    }
    if (rank >= r.top_groups) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = -INFINITY;
    }
  }
  // K rounds: the largest key of the warp, the lowest id among equal ones
  uint32_t taken = 0;
  e_lane = 0;
  bool open = false;
  for (int j = 0; j < r.K; ++j) {
    uint32_t best = 0;
    int best_e = 0x7fffffff, best_i = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = select_expert(r, lane, i);
      const uint32_t k = e < 0 || (taken >> i & 1) ? 0u : order_bits(v[i]);
      if (k > best) {
        best = k;
        best_e = e;
        best_i = i;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int e = __reduce_min_sync(0xffffffffu, best == top ? best_e : 0x7fffffff);
    if (best == top && best_e == e) taken |= 1u << best_i;
    if (lane == j) {
      e_lane = e;
      open = top > order_bits(-INFINITY);
    }
  }
  float s = 0.0f;
  if (lane < r.K && open) {
    const float l = logit(e_lane);
    s = r.sigmoid ? sigmoid_ieee(l) : expf(l - m) / total;
  }
  if (r.renormalize) s = s / (sum_lanes(s) + SELECT_SUM_EPS);
  w_lane = s * r.scale;
}

}  // namespace moe
