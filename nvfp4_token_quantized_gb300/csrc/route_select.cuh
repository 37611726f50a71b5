// route_select.cuh - the choice of experts of one token by one warp: scores,
// balance bias, groups, top-k, renormalised weights.  Used by the standalone
// kernel (kernels_select.cu) and the small-batch front kernel
// (kernels_route.cu).
//
// A row of 256 experts and 8 slots costs a few hundred instructions a warp
// while its bytes take the memory system far less, so what bounds the choice
// is instructions.  The usual row takes this path, several rows of a warp
// together:
//  - scores by the hardware's exponential and reciprocal;
//  - the two best of each lane (three where groups leave fewer lanes) and, with
//    groups, the two best of each group, by min and max;
//  - K rounds of a maximum over the lanes' heads, each lane moving on to its
//    next best.  If exactly K experts reach the last maximum, no two lanes
//    tied and none held one more: the rounds are the slots;
//  - the slots of all rows, one a lane: their scores at full accuracy, and the
//    weights.
// Comparisons, selections and logic take two issue slots a warp, additions and
// fused multiply-adds one: counts, ranks and the places of a lane's best are
// therefore sums of reaches(), not bit masks.
// Otherwise the experts that reach the last maximum, if at most 32, are
// ranked one a lane; and rows that this does not cover either (NaN, infinite
// scores or biases, fewer open experts than slots, many equal values) go
// through select_by_rounds.
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
      const int e = select_expert(r, lane, i);
      v[i] = s + (bias && e >= 0 ? __ldg(bias + e) : 0.0f);
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
        b1 = r.sigmoid ? sigmoid_ieee(b1) : expf(b1 - m);
        b2 = r.sigmoid ? sigmoid_ieee(b2) : expf(b2 - m);
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


// Scratch of one warp for RB rows.
template <int RB>
struct alignas(16) SelectScratch {  // (read 16 bytes at a time)
  int slot_e[RB][32];              // of the slots: lane << 5 | place, or a ranked row's experts
  float slot_s[32];                // a ranked row's scores
  uint32_t key[32];                // a ranked row's candidates: what they are compared by
  int e[32];                       // and their experts
  uint32_t reach[RB][32];          // each lane's experts that reach a row's bound
  float top[RB], total[RB];        // softmax: the largest logit, the sum
};

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

// The sum over the warp of one value a row; lane l gets row
// row_of_lane(l % 4 or 2)'s.  Each step hands half of the rows to the other
// half of the lanes; the order of additions is the same for every RB.
template <int RB>
__device__ __forceinline__ constexpr int row_of_lane(int l) {
  return RB == 4 ? 2 * (l & 1) + (l >> 1 & 1) : RB == 2 ? l & 1 : 0;
}
template <int RB>
__device__ __forceinline__ float sum_rows(const float (&v)[RB], int lane) {
  constexpr unsigned all = 0xffffffffu;
  const bool odd = lane & 1, high = lane & 2;
  float mine;
  if constexpr (RB == 4) {
    const float a = (odd ? v[2] : v[0]) + __shfl_xor_sync(all, odd ? v[0] : v[2], 1);
    const float b = (odd ? v[3] : v[1]) + __shfl_xor_sync(all, odd ? v[1] : v[3], 1);
    mine = (high ? b : a) + __shfl_xor_sync(all, high ? a : b, 2);
  } else {
    if constexpr (RB == 2) mine = (odd ? v[1] : v[0]) + __shfl_xor_sync(all, odd ? v[0] : v[1], 1);
    else mine = v[0] + __shfl_xor_sync(all, v[0], 1);
    mine += __shfl_xor_sync(all, mine, 2);
  }
#pragma unroll
  for (int o = 16; o > 2; o >>= 1) mine += __shfl_xor_sync(all, mine, o);
  return mine;
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

// The two or three best (DEPTH) of NE values, each as often as it occurs, by
// merging sorted runs: the k-th of two runs is the largest min(a_i, b_j) with
// i + j = k, a_0 and b_0 taken as infinite.
template <int NE, int DEPTH>
__device__ __forceinline__ void lane_best(const float (&v)[NE], float (&b)[DEPTH]) {
#pragma unroll
  for (int i = 0; i < NE; i += 4) {
    const float p1 = fmaxf(v[i], v[i + 1]), p2 = fminf(v[i], v[i + 1]);
    const float q1 = fmaxf(v[i + 2], v[i + 3]), q2 = fminf(v[i + 2], v[i + 3]);
    const float c1 = fmaxf(p1, q1), c2 = fmaxf(fmaxf(p2, q2), fminf(p1, q1));
    const float c3 = DEPTH > 2 ? fmaxf(fminf(p1, q2), fminf(p2, q1)) : 0.0f;
    if (i == 0) {
      b[0] = c1, b[1] = c2;
      if constexpr (DEPTH > 2) b[2] = c3;
    } else {
      if constexpr (DEPTH > 2) b[2] = fmaxf(fmaxf(fmaxf(b[2], c3), fminf(b[0], c2)), fminf(b[1], c1));
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

// What a kernel is compiled for: the score, what the choice compares, and
// whether groups limit it; SELECT_ANY asks the rule.
constexpr int SELECT_SIGMOID = 1, SELECT_BY_SCORE = 2, SELECT_LIMITED = 4, SELECT_ANY = -1;

// The choice for `valid` <= RB rows by one warp.  Row q's logits start
// q * stride elements on, its ids and weights go to ids / w + q * K.
template <int NE, int RB, int MODE>
__device__ __forceinline__ void select_rows(const RouteRule& r, const void* rows, int dtype, int64_t stride, int valid,
                                            const float* bias, const float (&b)[NE], bool bias_finite, int lane,
                                            SelectScratch<RB>& sm, int32_t* ids, float* w) {
  static_assert(RB == 1 || RB == 2 || RB == 4, "rows in pairs");
  constexpr unsigned all = 0xffffffffu;
  const bool sigmoid = MODE < 0 ? r.sigmoid != 0 : (MODE & SELECT_SIGMOID) != 0;
  const bool by_score = MODE < 0 ? r.by_score != 0 : (MODE & SELECT_BY_SCORE) != 0;
  const bool limited = MODE < 0 ? r.top_groups < r.groups : (MODE & SELECT_LIMITED) != 0;
  const bool need_total = !sigmoid && (by_score || !r.renormalize);
  const int lanes = 1 << r.lane_shift, g = lane >> r.lane_shift;
  unsigned odd = bias_finite ? 0u : (1u << valid) - 1u;  // rows for select_by_rounds

  float v[RB][NE];
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    if (q < valid) {
      load_logits<NE>(r, row_at(rows, dtype, q * stride), dtype, lane, v[q]);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[q][i] = -INFINITY;
    }
  }
  // this lane's best, and its group's score
  constexpr int DEPTH = MODE < 0 || (MODE & SELECT_LIMITED) ? 3 : 2;
  float best[RB][DEPTH], group[RB], part[RB], top[RB];
  auto without_id = [&](float f) {
    return dtype == MOE_DTYPE_F32 ? f : __uint_as_float(__float_as_uint(f) & ~0x1fffu);
  };
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    // A finite sum means finite logits.  Otherwise some are closed (fine), or
    // NaN or +inf, which select_by_rounds sorts out.
    float2 x = make_float2(v[q][0], v[q][1]);
#pragma unroll
    for (int i = 2; i < NE; i += 2) x = add2(x, make_float2(v[q][i], v[q][i + 1]));
    const bool closed = __any_sync(all, !(fabsf(x.x + x.y) < INFINITY));
    if (closed) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < NE; ++i) bad |= !(v[q][i] < INFINITY);
      if (__any_sync(all, bad)) odd |= 1u << q;
    }
    part[q] = top[q] = 0.0f;
    if (sigmoid ? by_score : need_total) {
      if (!sigmoid) {
        float m = v[q][0];
#pragma unroll
        for (int i = 1; i < NE; ++i) m = fmaxf(m, v[q][i]);
        m = warp_top(m);
        top[q] = m == -INFINITY ? 0.0f : m;
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float s = sigmoid ? sigmoid_fast(v[q][i]) + b[i] : exp_fast(v[q][i] - top[q]);
        part[q] += s;
        if (by_score && (!closed || v[q][i] != -INFINITY)) v[q][i] = s;
      }
    }
  }
  if (need_total) {
    // sums over the experts; a lane goes on with one of the rows
    float total = sum_rows<RB>(part, lane);
    if (total == 0.0f) total = 1.0f;
    if (lane < RB) sm.total[row_of_lane<RB>(lane)] = total;
    if (by_score) {
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        const float k = 1.0f / __shfl_sync(all, total, row_of_lane<RB>(q));  // (its own inverse)
#pragma unroll
        for (int i = 0; i < NE; ++i) v[q][i] = fmaf(v[q][i], k, b[i]);  // (-inf stays)
      }
    }
  } else if (!sigmoid && lane < RB) {
    // The sum cancels from renormalised weights (the best logit is among the
    // chosen, so their sum is far above the 1e-20).
    sm.total[lane] = 1.0f;
  }
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    if (!by_score && dtype != MOE_DTYPE_F32) {
      // Equal logits are common in 16 bits.  Their FP32 values end in 13 zero
      // bits or more: the expert's id there makes each its own, the lower id
      // the larger value.
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float f = v[q][i] + 0.0f;  // (-0 to +0)
        const unsigned id = g * r.size + select_place(r, lane, i);
        const unsigned bits = __float_as_uint(f) | (f < 0.0f ? id : id ^ 511u);
        if (f > -INFINITY) v[q][i] = __uint_as_float(bits);
      }
    }
    lane_best<NE, DEPTH>(v[q], best[q]);
    if (!sigmoid && !need_total) {
      const float m = without_id(warp_top(best[q][0]));
      top[q] = m == -INFINITY ? 0.0f : m;
    }
    if (!sigmoid && lane == 0) sm.top[q] = top[q];
    if (limited) {
      float b1 = best[q][0], b2 = best[q][1];
#pragma unroll
      for (int s = 0; s < 5; ++s)
        if (s < r.lane_shift) merge2(b1, b2, __shfl_xor_sync(all, b1, 1 << s), __shfl_xor_sync(all, b2, 1 << s));
      group[q] = b1;
      if (r.top2) {
        if (!by_score) {
          b1 = without_id(b1), b2 = without_id(b2);
          // (of a softmax, what its sum would divide)
          const float s1 = sigmoid ? sigmoid_fast(b1) : exp_fast(b1 - top[q]);
          const float s2 = sigmoid ? sigmoid_fast(b2) : exp_fast(b2 - top[q]);
          group[q] = b1 > -INFINITY ? s1 + s2 : -INFINITY;
        } else if (b2 > -INFINITY) {
          group[q] = b1 + b2;
        }
      }
    }
  }
  // Which groups each row keeps.  A group's score is in all its lanes: lane d
  // of a group ranks the groups of row d, all rows at once.  (Every lane takes
  // part, also those of groups past the last one, whose score of -inf at a
  // higher index outranks none.)
  unsigned kept = all;  // bit of lane (group's first + d): row d keeps the group
  const bool together = lanes >= RB;
  auto rank_of = [&](float mine) {
    float rank = 0.0f;
    const int others = 32 >> r.lane_shift;
#pragma unroll
    for (int k = 1; k < 32; ++k) {
      if (k >= others) break;
      // (an equal score at a lower index outranks; of groups without an open
      // expert it does not matter which are kept)
      rank += reaches(__shfl_xor_sync(all, mine, k << r.lane_shift), mine, (g ^ k) < g ? 1.0f : 0.0f);
    }
    return rank;
  };
  const float top_groups = (float)r.top_groups;
  if (limited && together) {
    float mine = group[0];
#pragma unroll
    for (int q = 1; q < RB; ++q) mine = (lane & (RB - 1)) == q ? group[q] : mine;
    const float rank = rank_of(mine);
    kept = __ballot_sync(all, g < r.groups && rank < top_groups);
  }
  // K rounds for all rows at once.  pops: the rounds this lane's best won, k
  // (from 1) as digits of base 64, the best's highest.
  float head[RB][DEPTH], low[RB];
  unsigned pops[RB];
  unsigned mine = 0;  // rows that keep this lane's group
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    bool keep = g < r.groups;
    if (limited) {
      if (together) {
        keep = kept >> ((lane & ~(lanes - 1)) + q) & 1;
      } else {
        const float rank = rank_of(group[q]);
        keep = keep && rank < top_groups;
      }
    }
    mine |= (unsigned)keep << q;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) head[q][d] = keep ? best[q][d] : -INFINITY;
    pops[q] = 0;
    low[q] = -INFINITY;
  }
#pragma unroll 1
  for (int k = 1; k <= r.K; ++k) {
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      low[q] = warp_top(head[q][0]);
      if (head[q][0] == low[q]) {
        pops[q] = pops[q] * 64 + k;
#pragma unroll
        for (int d = 0; d + 1 < DEPTH; ++d) head[q][d] = head[q][d + 1];
        head[q][DEPTH - 1] = -INFINITY;
      }
    }
  }
  unsigned ranked = 0;  // rows whose candidates are to be ranked
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    // How many of this lane's reach the last maximum (every open expert of the
    // kept groups where the heads ran out), the sum of their places, and the
    // place of its best.
    const bool keep = mine >> q & 1;
    const float bound = keep ? fmaxf(low[q], -3.402823466e38f) : INFINITY;
    float both_sums = 0.0f, first = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      both_sums = fmaf(reaches(v[q][i], bound), (float)(1 + 64 * i), both_sums);
      first = fmaf(reaches(v[q][i], best[q][0]), (float)i, first);
    }
    const int count = whole(both_sums) & 63, places = whole(both_sums) >> 6;
    const int n = __reduce_add_sync(all, count);
    if (n < r.K || n > 32) odd |= 1u << q;
    // Settled if the last maximum is an open expert's and K experts reach it:
    // each is one of its lane's best and won a round of its own.  Their places
    // follow from the sums, if no two of a lane's are equal.
    const bool twice = (best[q][1] >= bound && best[q][0] == best[q][1]) ||
                       (DEPTH > 2 && best[q][DEPTH - 1] >= bound && best[q][1] == best[q][DEPTH - 1]);
    float least = fminf(fabsf(bound), limited ? fabsf(group[q]) : INFINITY);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) least = fminf(least, fabsf(best[q][d]));
    const bool unsafe = least < TINY;
    bool settles = n == r.K && low[q] > -INFINITY;
    if (__any_sync(all, twice || unsafe)) {
      settles = false;
      if (__any_sync(all, unsafe)) odd |= 1u << q;
    }
    if (q >= valid || (odd >> q & 1)) continue;
    if (settles) {
      // slots hold lane and place; the best won the first of the lane's rounds
      const int here = lane << 5, best_at = whole(first);
      if (count > 0) sm.slot_e[q][(pops[q] >> 6 * (count - 1)) - 1] = here + best_at;
      if (count == 2) sm.slot_e[q][(pops[q] & 63) - 1] = here + places - best_at;
      if (DEPTH > 2 && __any_sync(all, count > 2)) {
        float second = 0.0f;  // places of the two best
#pragma unroll
        for (int i = 0; i < NE; ++i) second = fmaf(reaches(v[q][i], best[q][1]), (float)i, second);
        if (count > 2) {
          sm.slot_e[q][(pops[q] >> 6 & 63) - 1] = here + whole(second) - best_at;
          sm.slot_e[q][(pops[q] & 63) - 1] = here + places - whole(second);
        }
      }
    } else {
      ranked |= 1u << q;
      unsigned reach = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) reach |= v[q][i] >= bound ? 1u << i : 0u;
      sm.reach[q][lane] = reach;
    }
  }
  const unsigned rows_here = (1u << valid) - 1u;
  odd &= rows_here;
  __syncwarp();
  // the slots of the rows that the rounds settled
  const unsigned settled = rows_here & ~odd & ~ranked;
  const int slots = 1 << r.slot_shift, at_once = 32 >> r.slot_shift;
  if (settled) {
#pragma unroll 1
    for (int q0 = 0; q0 < RB; q0 += at_once) {
      const int q = q0 + (lane >> r.slot_shift), c = lane & (slots - 1);
      const bool slot = q < RB && (settled >> q & 1) && c < r.K;
      float s = 0.0f;
      int e = 0;
      if (slot) {
        const int x = sm.slot_e[q][c];  // lane and place
        e = (x >> 5 >> r.lane_shift) * r.size + select_place(r, x >> 5, x & 31);
        const float l = logit_at(row_at(rows, dtype, q * stride), dtype, e);
        s = sigmoid ? sigmoid_ieee(l) : expf(l - sm.top[q]) / sm.total[q];
      }
      if (r.renormalize) {
        float sum = s;
#pragma unroll 1
        for (int o = slots >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(all, sum, o);
        s = s / (sum + SELECT_SUM_EPS);
      }
      if (slot) {
        ids[q * r.K + c] = e;
        w[q * r.K + c] = s * r.scale;
      }
    }
  }
  // rows with ties or a lane with three: the candidates, one a lane
  while (ranked) {
    const int q = __ffs(ranked) - 1;
    ranked &= ranked - 1;
    const void* row = row_at(rows, dtype, q * stride);
    unsigned reach = sm.reach[q][lane];
    int upto = __popc(reach);
    int at = -upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(all, upto, o);
      if (lane >= o) upto += t;
    }
    const int n = __shfl_sync(all, upto, 31);
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
    int e = 0;
    if (lane < n) {
      e = sm.e[lane];
      const float l = logit_at(row, dtype, e);
      float value = l;
      score = sigmoid ? sigmoid_ieee(l) : expf(l - sm.top[q]) / sm.total[q];
      if (by_score) value = score + (bias ? __ldg(bias + e) : 0.0f);
      key = order_bits(value);
    }
    sm.key[lane] = key;
    __syncwarp();
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&sm.key[j]);
      const int4 oe = *reinterpret_cast<const int4*>(&sm.e[j]);
      rank += o.x > key || (o.x == key && oe.x < e);
      rank += o.y > key || (o.y == key && oe.y < e);
      rank += o.z > key || (o.z == key && oe.z < e);
      rank += o.w > key || (o.w == key && oe.w < e);
    }
    if (lane < n && rank < r.K) {
      sm.slot_s[rank] = score;
      sm.slot_e[q][rank] = e;
    }
    __syncwarp();
    float s = lane < r.K ? sm.slot_s[lane] : 0.0f;
    if (r.renormalize) s = s / (sum_lanes(s) + SELECT_SUM_EPS);
    if (lane < r.K) {
      ids[q * r.K + lane] = sm.slot_e[q][lane];
      w[q * r.K + lane] = s * r.scale;
    }
    __syncwarp();
  }
  // the rows left over
  while (odd) {
    const int q = __ffs(odd) - 1;
    odd &= odd - 1;
    const void* row = row_at(rows, dtype, q * stride);
    float raw[NE];
    load_logits<NE>(r, row, dtype, lane, raw);
    int e;
    float wj;
    select_by_rounds<NE>(r, row, dtype, bias, lane, raw, e, wj);
    if (lane < r.K) {
      ids[q * r.K + lane] = e;
      w[q * r.K + lane] = wj;
    }
  }
  __syncwarp();
}

}  // namespace moe
