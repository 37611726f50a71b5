// route_select.cuh - the choice of experts of one token by one warp: scores,
// balance bias, groups, top-k, renormalised weights.  Used by the kernel for
// small batches (kernels_select.cu), where latency counts, and the fused front
// of a small forward (kernels_route.cu); larger batches take select_parts.cuh,
// which gives the same bits.
//
// Instructions bound it, a chain of some hundreds:
//  - scores by the hardware's exponential and reciprocal;
//  - the three best of each lane and, with groups, the two best of each group,
//    by min and max;
//  - K rounds of a maximum over the lanes' heads, each lane moving on to its
//    next best.  If exactly K experts reach the last maximum, no two lanes
//    tied and none held one more: the rounds are the slots, whose scores are
//    then taken at full accuracy.
// Comparisons, selections and logic take two issue slots a warp, additions and
// fused multiply-adds one: counts, ranks and the places of a lane's best are
// therefore sums of reaches(), not bit masks.
// Otherwise the experts that reach the last maximum, if at most 32, are
// ranked one a lane; and rows that this does not cover either (NaN, infinite
// scores or biases, fewer open experts than slots, many equal values) go
// through select_by_rounds, behind which a grid of few waves ends (4073 x 128 bf16
// with padding tokens: 6.4 us, 4.6 without them at 4096).
#pragma once

#include "common.cuh"
#include "elem_types.cuh"
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

// exp(x) and 1 / (1 + exp(-x)) for the choice: relative errors of a few
// 2^-24 and absolute ones under 2e-7.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + exp_fast(-x)));
  return y;
}

// A sum of up to 512 values of [0, 1] that does not depend on their order, so
// that a row's weights do not depend on how many rows a call has: each value
// is split into a multiple of 2^-14 and one of 2^-29 (what is left, under
// 2^-30, is dropped), whose sums are exact in FP32.
struct OrderFree {
  float2 high = {0.0f, 0.0f}, low = {0.0f, 0.0f};
  __device__ __forceinline__ void add(float2 e) {
    const float2 h = add2(add2(e, both(768.0f)), both(-768.0f));
    const float2 rest = fma2(h, both(-1.0f), e);
    high = add2(high, h);
    low = add2(low, add2(add2(rest, both(0.0234375f)), both(-0.0234375f)));
  }
  // of the warp's lanes
  __device__ __forceinline__ float over_warp() const {
    const int h = __reduce_add_sync(0xffffffffu, __float2int_rn((high.x + high.y) * 16384.0f));
    const int l = __reduce_add_sync(0xffffffffu, __float2int_rn((low.x + low.y) * 536870912.0f));
    return fmaf((float)l, 1.0f / 536870912.0f, (float)h * (1.0f / 16384.0f));
  }
};

// The place of local slot i of this lane in its group, and its expert or -1.
__device__ __forceinline__ int select_place(const RouteRule& r, int lane, int i) {
  const int lanes = 1 << r.lane_shift, l = lane & (lanes - 1);
  return r.vec ? ((i >> 2) * lanes + l) * 4 + (i & 3) : i * lanes + l;
}
__device__ __forceinline__ int select_expert(const RouteRule& r, int lane, int i) {
  const int g = lane >> r.lane_shift, o = select_place(r, lane, i);
  return g < r.groups && o < r.size ? g * r.size + o : -1;
}

// Logit e of a row of moe_dtype `dtype`.
__device__ __forceinline__ float logit_at(const void* row, int dtype, int e) {
  if (dtype == MOE_DTYPE_F32) return static_cast<const float*>(row)[e];
  if (dtype == MOE_DTYPE_F16) return to_f32(static_cast<const __half*>(row)[e]);
  return to_f32(static_cast<const __nv_bfloat16*>(row)[e]);
}
__device__ __forceinline__ const void* row_at(const void* rows, int dtype, int64_t elements) {
  return static_cast<const char*>(rows) + elements * (dtype == MOE_DTYPE_F32 ? 4 : 2);
}

// Any row, one at a time: K rounds that each take the largest value of the
// warp.  raw[i]: the logit of this lane's expert i (-inf where it has none).
// Lane j < K returns slot j in e_lane and w_lane.  All 32 lanes call it.
template <int NE>
__device__ __noinline__ void select_by_rounds(const RouteRule& r, const void* row, int dtype, const float* bias,
                                              int lane, const float (&raw)[NE], int& e_lane, float& w_lane) {
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
      OrderFree sum;
#pragma unroll
      for (int i = 0; i < NE; i += 2) sum.add(make_float2(exp_fast(raw[i] - m), exp_fast(raw[i + 1] - m)));
      total = sum.over_warp();
      if (total == 0.0f) total = 1.0f;
    }
  }
  // what the choice compares; -inf: closed
  const float k = 1.0f / total;
  float v[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    v[i] = raw[i];
    if (r.by_score && raw[i] != -INFINITY) {
      const int e = select_expert(r, lane, i);
      const float b = bias && e >= 0 ? __ldg(bias + e) : 0.0f;
      v[i] = r.sigmoid ? sigmoid_fast(raw[i]) + b : fmaf(exp_fast(raw[i] - m), k, b);
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
    float gs = b1;
    if (r.top2 && b1 > -INFINITY) {
      // (of a softmax, what its sum would divide)
      if (!r.by_score) {
        b1 = r.sigmoid ? sigmoid_fast(b1) : exp_fast(b1 - m);
        b2 = r.sigmoid ? sigmoid_fast(b2) : exp_fast(b2 - m);
      }
      gs = b2 > -INFINITY ? b1 + b2 : b1;
    }
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
    const float l = logit_at(row, dtype, e_lane);
    s = r.sigmoid ? sigmoid_ieee(l) : expf(l - m) / total;
  }
  if (r.renormalize) s = s / (sum_lanes(s) + SELECT_SUM_EPS);
  w_lane = s * r.scale;
}


// Shared memory of a warp's row.
struct alignas(16) SelectScratch {  // (read 16 bytes at a time)
  uint32_t key[32];  // candidates: what they are compared by
  int e[32];         // and their experts
  int slot_e[32];    // the slots' experts
  float slot_s[32];  // and scores
};

// The largest over the warp.
__device__ __forceinline__ float warp_top(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// 1 where v >= bound, else 0 (a = 1); 1 only where v > bound with a = 0; 0
// where v - bound is NaN.  Exact unless the two differ by less than 2^-126,
// which takes a bound below TINY: the caller sends such rows another way.
constexpr float TINY = 7.888609e-31f;  // 2^-100
__device__ __forceinline__ float reaches(float v, float bound, float a = 1.0f) {
  return __saturatef(fmaf(v - bound, 8.507059173e37f, a));
}
// A small non-negative whole float as an integer.
__device__ __forceinline__ int whole(float v) { return __float_as_int(v + 8388608.0f) & 0x7fffff; }

// Merges the two best (b1 >= b2) of two sets.
__device__ __forceinline__ void merge2(float& b1, float& b2, float c1, float c2) {
  b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
  b1 = fmaxf(b1, c1);
}

// The logits of this lane's experts, -inf where it has none.
template <int NE>
__device__ __forceinline__ void load_logits(const RouteRule& r, const void* row, int dtype, int lane,
                                            float (&raw)[NE]) {
  const int lanes = 1 << r.lane_shift;
  const int g = lane >> r.lane_shift, l = lane & (lanes - 1);
  const int size = g < r.groups ? r.size : 0;
  if (r.vec) {
    const int at = g * r.size + l * 4;
#pragma unroll
    for (int c = 0; c < NE / 4; ++c) {
#pragma unroll
      for (int k = 0; k < 4; ++k) raw[4 * c + k] = -INFINITY;
      if ((c * lanes + l) * 4 < size) {
        const int e = at + c * lanes * 4;
        if (dtype == MOE_DTYPE_F32) {
          const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + e);
          raw[4 * c] = f.x, raw[4 * c + 1] = f.y, raw[4 * c + 2] = f.z, raw[4 * c + 3] = f.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + e);
          const bool half = dtype == MOE_DTYPE_F16;
          const float2 a = half ? unpack2(q.x, __half()) : unpack2(q.x, __nv_bfloat16());
          const float2 b = half ? unpack2(q.y, __half()) : unpack2(q.y, __nv_bfloat16());
          raw[4 * c] = a.x, raw[4 * c + 1] = a.y, raw[4 * c + 2] = b.x, raw[4 * c + 3] = b.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      raw[i] = i * lanes + l < size ? logit_at(row, dtype, g * r.size + l + i * lanes) : -INFINITY;
  }
}

// The three best of NE values, each as often as it occurs, by merging sorted
// runs: the k-th of two runs is the largest min(a_i, b_j) with i + j = k, a_0
// and b_0 taken as infinite.
template <int NE>
__device__ __forceinline__ void lane_best(const float (&v)[NE], float (&b)[3]) {
#pragma unroll
  for (int i = 0; i < NE; i += 4) {
    const float p1 = fmaxf(v[i], v[i + 1]), p2 = fminf(v[i], v[i + 1]);
    const float q1 = fmaxf(v[i + 2], v[i + 3]), q2 = fminf(v[i + 2], v[i + 3]);
    const float c1 = fmaxf(p1, q1), c2 = fmaxf(fmaxf(p2, q2), fminf(p1, q1));
    const float c3 = fmaxf(fminf(p1, q2), fminf(p2, q1));
    if (i == 0) {
      b[0] = c1, b[1] = c2, b[2] = c3;
    } else {
      b[2] = fmaxf(fmaxf(fmaxf(b[2], c3), fminf(b[0], c2)), fminf(b[1], c1));
      b[1] = fmaxf(fmaxf(b[1], c2), fminf(b[0], c1));
      b[0] = fmaxf(b[0], c1);
    }
  }
}

// The balance bias of this lane's experts; returns whether all are finite.
template <int NE>
__device__ __forceinline__ bool load_bias(const RouteRule& r, const float* bias, int lane, float (&b)[NE]) {
  float x = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = select_expert(r, lane, i);
    b[i] = bias && e >= 0 ? __ldg(bias + e) : 0.0f;
    x += fabsf(b[i]);
  }
  return __all_sync(0xffffffffu, x < INFINITY);
}

// The choice for one row by one warp, for its latency.  b: the balance bias
// of this lane's experts.
template <int NE>
__device__ __forceinline__ void select_row(const RouteRule& r, const void* row, int dtype, const float* bias,
                                           const float (&b)[NE], bool bias_finite, int lane, SelectScratch& sm,
                                           int32_t* ids, float* w) {
  constexpr unsigned all = 0xffffffffu;
  const bool sigmoid = r.sigmoid, by_score = r.by_score, limited = r.top_groups < r.groups;
  const bool need_total = !sigmoid && (by_score || !r.renormalize);
  const int lanes = 1 << r.lane_shift, g = lane >> r.lane_shift;

  float v[NE];
  load_logits<NE>(r, row, dtype, lane, v);
  // A finite sum means finite logits.  Otherwise some are closed (fine), or
  // NaN or +inf, which select_by_rounds sorts out.
  bool odd = !bias_finite;  // for select_by_rounds
  float2 x = make_float2(v[0], v[1]);
#pragma unroll
  for (int i = 2; i < NE; i += 2) x = add2(x, make_float2(v[i], v[i + 1]));
  const bool closed = __any_sync(all, !(fabsf(x.x + x.y) < INFINITY));
  if (closed) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NE; ++i) bad |= !(v[i] < INFINITY);
    odd |= __any_sync(all, bad) != 0;
  }
  float top = 0.0f, total = 1.0f, k = 1.0f;
  if (sigmoid && by_score) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float s = sigmoid_fast(v[i]) + b[i];
      if (!closed || v[i] != -INFINITY) v[i] = s;
    }
  }
  if (need_total) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) m = fmaxf(m, v[i]);
    m = warp_top(m);
    top = m == -INFINITY ? 0.0f : m;
    OrderFree sum;
#pragma unroll
    for (int i = 0; i < NE; i += 2) {
      const float2 e = make_float2(exp_fast(v[i] - top), exp_fast(v[i + 1] - top));
      sum.add(e);
      if (by_score && (!closed || v[i] != -INFINITY)) v[i] = e.x;
      if (by_score && (!closed || v[i + 1] != -INFINITY)) v[i + 1] = e.y;
    }
    total = sum.over_warp();
    if (total == 0.0f) total = 1.0f;
    if (by_score) {
      k = 1.0f / total;
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = fmaf(v[i], k, b[i]);  // (-inf stays)
    }
  }
  if (!by_score && dtype != MOE_DTYPE_F32) {
    // Equal logits are common in 16 bits.  Their FP32 values end in 13 zero
    // bits or more: the expert's id there makes each its own, the lower id
    // the larger value.
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float f = v[i] + 0.0f;  // (-0 to +0)
      const unsigned id = g * r.size + select_place(r, lane, i);
      const unsigned bits = __float_as_uint(f) | (f < 0.0f ? id : id ^ 511u);
      if (f > -INFINITY) v[i] = __uint_as_float(bits);
    }
  }
  auto without_id = [&](float f) {
    return dtype == MOE_DTYPE_F32 ? f : __uint_as_float(__float_as_uint(f) & ~0x1fffu);
  };
  // this lane's best three, and its group's score
  float best[3];
  lane_best<NE>(v, best);
  if (!sigmoid && !need_total) {
    // (The sum cancels from renormalised weights: the best logit is among the
    // chosen, so their sum is far above the 1e-20.)
    const float m = without_id(warp_top(best[0]));
    top = m == -INFINITY ? 0.0f : m;
  }
  bool keep = g < r.groups;
  float group = INFINITY;
  if (limited) {
    float b1 = best[0], b2 = best[1];
#pragma unroll
    for (int s = 0; s < 5; ++s)
      if (s < r.lane_shift) merge2(b1, b2, __shfl_xor_sync(all, b1, 1 << s), __shfl_xor_sync(all, b2, 1 << s));
    group = b1;
    if (r.top2) {
      if (!by_score) {
        b1 = without_id(b1), b2 = without_id(b2);
        // (of a softmax, what its sum would divide)
        const float s1 = sigmoid ? sigmoid_fast(b1) : exp_fast(b1 - top);
        const float s2 = sigmoid ? sigmoid_fast(b2) : exp_fast(b2 - top);
        group = b1 > -INFINITY ? s1 + s2 : -INFINITY;
      } else if (b2 > -INFINITY) {
        group = b1 + b2;
      }
    }
    // Its rank.  (Every lane takes part, also those of groups past the last
    // one, whose score of -inf at a higher index outranks none.)
    float rank = 0.0f;
    const int others = 32 >> r.lane_shift;
#pragma unroll
    for (int j = 1; j < 32; ++j) {
      if (j >= others) break;
      // (an equal score at a lower index outranks; of groups without an open
      // expert it does not matter which are kept)
      rank += reaches(__shfl_xor_sync(all, group, j << r.lane_shift), group, (g ^ j) < g ? 1.0f : 0.0f);
    }
    keep = keep && rank < (float)r.top_groups;
  }
  // K rounds.  pops: the rounds this lane's best won, as digits of base 64
  // (from 1), the best's highest.
  float h0 = keep ? best[0] : -INFINITY, h1 = keep ? best[1] : -INFINITY, h2 = keep ? best[2] : -INFINITY;
  float low = -INFINITY;
  unsigned pops = 0;
#pragma unroll 1
  for (int j = 1; j <= r.K; ++j) {
    low = warp_top(h0);
    if (h0 == low) {
      pops = pops * 64 + j;
      h0 = h1, h1 = h2, h2 = -INFINITY;
    }
  }
  // How many of this lane's reach the last maximum (every open expert of the
  // kept groups where the heads ran out), the sum of their places, and the
  // place of its best.
  const float bound = keep ? fmaxf(low, -3.402823466e38f) : INFINITY;
  float both_sums = 0.0f, first = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    both_sums = fmaf(reaches(v[i], bound), (float)(1 + 64 * i), both_sums);
    first = fmaf(reaches(v[i], best[0]), (float)i, first);
  }
  const int count = whole(both_sums) & 63, places = whole(both_sums) >> 6;
  int n = __reduce_add_sync(all, count);
  // Settled if the last maximum is an open expert's and K experts reach it:
  // each is one of its lane's best and won a round of its own.  Their places
  // follow from the sums, if no two of a lane's are equal.
  const bool twice = (best[1] >= bound && best[0] == best[1]) || (best[2] >= bound && best[1] == best[2]);
  float least = fminf(fabsf(bound), fabsf(group));
  least = fminf(fminf(least, fabsf(best[0])), fminf(fabsf(best[1]), fabsf(best[2])));
  const bool tied = __any_sync(all, twice);
  odd |= __any_sync(all, least < TINY) || n < r.K || n > 32;
  if (odd) {
    float raw[NE];
    load_logits<NE>(r, row, dtype, lane, raw);
    int e;
    float wj;
    select_by_rounds<NE>(r, row, dtype, bias, lane, raw, e, wj);
    if (lane < r.K) {
      ids[lane] = e;
      w[lane] = wj;
    }
    return;
  }
  auto score_of = [&](float l) { return sigmoid ? sigmoid_ieee(l) : expf(l - top) / total; };
  int e = 0;
  float s = 0.0f;
  if (n == r.K && low > -INFINITY && !tied) {
    // slots hold experts; the best won the first of the lane's rounds
    const int best_at = whole(first);
    auto expert = [&](int place) { return g * r.size + select_place(r, lane, place); };
    if (count > 0) sm.slot_e[(pops >> 6 * (count - 1)) - 1] = expert(best_at);
    if (count == 2) sm.slot_e[(pops & 63) - 1] = expert(places - best_at);
    if (__any_sync(all, count > 2)) {
      float second = 0.0f;  // places of the two best
#pragma unroll
      for (int i = 0; i < NE; ++i) second = fmaf(reaches(v[i], best[1]), (float)i, second);
      if (count > 2) {
        sm.slot_e[(pops >> 6 & 63) - 1] = expert(whole(second) - best_at);
        sm.slot_e[(pops & 63) - 1] = expert(places - whole(second));
      }
    }
    __syncwarp();
    if (lane < r.K) {
      e = sm.slot_e[lane];
      s = score_of(logit_at(row, dtype, e));
    }
  } else {
    // ties, or a lane with more: the candidates, one a lane
    unsigned reach = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) reach |= v[i] >= bound ? 1u << i : 0u;
    int upto = __popc(reach);
    int at = -upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(all, upto, o);
      if (lane >= o) upto += t;
    }
    n = __shfl_sync(all, upto, 31);
    at += upto;
    while (reach) {
      const int i = __ffs(reach) - 1;
      reach &= reach - 1;
      sm.e[at++] = g * r.size + select_place(r, lane, i);
    }
    __syncwarp();
    // they compare as (value, lower id first)
    float score = 0.0f;
    uint32_t key = 0;
    int mine = 0;
    if (lane < n) {
      mine = sm.e[lane];
      const float l = logit_at(row, dtype, mine);
      float value = l;
      score = score_of(l);
      if (by_score) {
        const float bb = bias ? __ldg(bias + mine) : 0.0f;
        value = sigmoid ? sigmoid_fast(l) + bb : fmaf(exp_fast(l - top), k, bb);
      }
      key = order_bits(value);
    }
    sm.key[lane] = key;
    __syncwarp();
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&sm.key[j]);
      const int4 oe = *reinterpret_cast<const int4*>(&sm.e[j]);
      rank += o.x > key || (o.x == key && oe.x < mine);
      rank += o.y > key || (o.y == key && oe.y < mine);
      rank += o.z > key || (o.z == key && oe.z < mine);
      rank += o.w > key || (o.w == key && oe.w < mine);
    }
    if (lane < n && rank < r.K) {
      sm.slot_s[rank] = score;
      sm.slot_e[rank] = mine;
    }
    __syncwarp();
    if (lane < r.K) {
      e = sm.slot_e[lane];
      s = sm.slot_s[lane];
    }
  }
  if (r.renormalize) s = s / (sum_lanes(s) + SELECT_SUM_EPS);
  if (lane < r.K) {
    ids[lane] = e;
    w[lane] = s * r.scale;
  }
  __syncwarp();
}

}  // namespace moe
