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
//  - the two best of each lane, block of lanes and group by min and max;
//  - a bound that at least K experts reach and few more: up to 8 slots the
//    lowest second best of the chosen groups' blocks, above the K-th of the
//    lanes' two best, by K rounds of a maximum over the warp;
//  - those candidates, one a lane, two rows side by side: their scores again
//    at full accuracy (for the weights), and the rank of each among them.
// Rows it does not cover (NaN, infinite scores or biases, fewer open experts
// than slots, more than 32 candidates, as with many equal values) go through
// select_by_rounds.
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
    const float l = logit_at(row, dtype, e_lane);
    s = r.sigmoid ? sigmoid_ieee(l) : expf(l - m) / total;
  }
  if (r.renormalize) s = s / (sum_lanes(s) + SELECT_SUM_EPS);
  w_lane = s * r.scale;
}


// Scratch of one warp for RB rows.
template <int RB>
struct SelectScratch {
  uint32_t key[RB][32];  // candidates: what they are compared by
  int e[RB][32];         // and their experts
  float out_s[RB][32];  // slots: scores
  int out_e[RB][32];    // and experts
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
  float top[RB], total[RB];  // softmax: the largest logit, the sum
  float lane1[RB], block2[RB], group[RB];
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
    top[q] = 0.0f, total[q] = 1.0f;
    if (!sigmoid) {
      float m = v[q][0];
#pragma unroll
      for (int i = 1; i < NE; ++i) m = fmaxf(m, v[q][i]);
      m = max_lanes(m);
      top[q] = m == -INFINITY ? 0.0f : m;
    }
    if (by_score || need_total) {
      float s[NE];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        s[i] = sigmoid ? sigmoid_fast(v[q][i]) : exp_fast(v[q][i] - top[q]);
        if (need_total) sum += s[i];
      }
      if (need_total) {
        sum = sum_lanes(sum);
        total[q] = sum == 0.0f ? 1.0f : sum;
      }
      if (by_score) {
        if (closed) {
#pragma unroll
          for (int i = 0; i < NE; ++i)
            if (v[q][i] == -INFINITY) s[i] = -INFINITY;
        }
        const float k = sigmoid ? 1.0f : 1.0f / total[q];
#pragma unroll
        for (int i = 0; i < NE; ++i) v[q][i] = sigmoid ? s[i] + b[i] : fmaf(s[i], k, b[i]);
      }
    }
    float b1 = fmaxf(v[q][0], v[q][1]), b2 = fminf(v[q][0], v[q][1]);
#pragma unroll
    for (int i = 2; i < NE; i += 2)
      merge2(b1, b2, fmaxf(v[q][i], v[q][i + 1]), fminf(v[q][i], v[q][i + 1]));
    lane1[q] = b1;
    auto merge_lanes = [&](int from, int to) {
#pragma unroll 1
      for (int s = from; s < to; ++s)
        merge2(b1, b2, __shfl_xor_sync(all, b1, 1 << s), __shfl_xor_sync(all, b2, 1 << s));
    };
    merge_lanes(0, r.block_shift);
    block2[q] = b2;
    if (limited) {
      merge_lanes(max(r.block_shift, 0), r.lane_shift);
      group[q] = r.top2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
  }
  // Which groups each row keeps.  A group's score is in all its lanes: lane d
  // of a group ranks the groups of row d, all rows at once.  (Every lane takes
  // part, also those of groups past the last one, whose score of -inf at a
  // higher index outranks none.)
  unsigned kept = all;  // bit of lane (group's first + d): row d keeps the group
  const bool together = lanes >= RB;
  auto rank_of = [&](float mine) {
    int rank = 0;
#pragma unroll 1
    for (int k = 1; k < (32 >> r.lane_shift); ++k) {
      const float other = __shfl_xor_sync(all, mine, k << r.lane_shift);
      rank += other > mine || (other == mine && (g ^ k) < g);
    }
    return rank;
  };
  if (limited && together) {
    float mine = group[0];
#pragma unroll
    for (int q = 1; q < RB; ++q) mine = (lane & (RB - 1)) == q ? group[q] : mine;
    const int rank = rank_of(mine);
    kept = __ballot_sync(all, g < r.groups && rank < r.top_groups);
  }
  // the candidates of each row: a bit for each of this lane's experts, and
  // how many the lower lanes have (a byte for each row)
  unsigned mask[RB];
  unsigned counts = 0;
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    bool keep = g < r.groups;
    if (limited) {
      if (together) {
        keep = kept >> ((lane & ~(lanes - 1)) + q) & 1;
      } else {
        const int rank = rank_of(group[q]);
        keep = keep && rank < r.top_groups;
      }
    }
    // the bound: the lowest second best of the kept blocks, or the K-th of the
    // two best of every kept lane (-inf where there are too few)
    uint32_t low;
    if (r.block_shift >= 0) {
      low = __reduce_min_sync(all, keep ? order_bits(block2[q]) : 0xffffffffu);
    } else {
      uint32_t head = keep ? order_bits(lane1[q]) : 0u, next = keep ? order_bits(block2[q]) : 0u;
#pragma unroll 1
      for (int k = 0; k < r.K; ++k) {
        low = __reduce_max_sync(all, head);
        if (head == low) {
          head = next;
          next = 0u;
        }
      }
    }
    float bound = low == 0u ? -INFINITY : __uint_as_float((low & 0x80000000u) ? (low & 0x7FFFFFFFu) : ~low);
    bound = keep ? fmaxf(bound, -3.402823466e38f) : __int_as_float(0x7fffffff);  // (NaN: none)
    mask[q] = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (v[q][i] >= bound) mask[q] |= 1u << i;
    counts |= (unsigned)__popc(mask[q]) << (8 * q);
  }
  // (bytes hold the counts of up to 255 candidates a row)
  unsigned upto = counts;
  if constexpr (NE * 32 > 255) {
    // more could carry into the next row's byte: saturate by giving rows with
    // many up beforehand
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const unsigned n = __reduce_add_sync(all, (unsigned)__popc(mask[q]));
      if (n > 255) {
        odd |= 1u << q;
        counts &= ~(255u << (8 * q));
      }
    }
    upto = counts;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(all, upto, o);
    if (lane >= o) upto += t;
  }
  const unsigned totals = __shfl_sync(all, upto, 31);
  upto -= counts;
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    const int n = totals >> (8 * q) & 255;
    if (n < r.K || n > 32) odd |= 1u << q;
    if ((odd >> q & 1) || q >= valid) continue;
    int at = upto >> (8 * q) & 255;
    while (mask[q]) {
      const int i = __ffs(mask[q]) - 1;
      mask[q] &= mask[q] - 1;
      sm.e[q][at++] = g * r.size + select_place(r, lane, i);
    }
  }
  odd &= (1u << valid) - 1u;
  __syncwarp();
  // The candidates, one a lane: two rows side by side where both fit.
#pragma unroll
  for (int q0 = 0; q0 < RB; q0 += 2) {
    constexpr int PAIR = RB > 1 ? 1 : 0;
    if (q0 >= valid) break;
    const int n0 = (odd >> q0 & 1) ? 0 : totals >> (8 * q0) & 255;
    const int n1 =
        PAIR == 0 || q0 + 1 >= valid || (odd >> (q0 + PAIR) & 1) ? 0 : totals >> (8 * (q0 + PAIR)) & 255;
    const bool paired = PAIR == 1 && n0 <= 16 && n1 <= 16 && r.K <= 16;
    for (int pass = 0; pass < (paired || PAIR == 0 ? 1 : 2); ++pass) {
      const bool second = paired ? lane >= 16 : pass == 1;
      const int q = q0 + (second ? PAIR : 0);
      const int n = second ? n1 : n0;
      const int c = paired ? lane & 15 : lane;
      const int longest = paired ? max(n0, n1) : n;
      float score = 0.0f;
      // candidates compare as (value, lower id first)
      uint32_t key = 0;
      int e = 0;
      if (c < n) {
        e = sm.e[q][c];
        const float l = logit_at(row_at(rows, dtype, q * stride), dtype, e);
        float value = l;
        if (sigmoid) score = sigmoid_ieee(l);
        else score = expf(l - (second ? top[q0 + PAIR] : top[q0])) / (second ? total[q0 + PAIR] : total[q0]);
        if (by_score) value = score + (bias ? __ldg(bias + e) : 0.0f);
        key = order_bits(value);
      }
      sm.key[q][c] = key;
      __syncwarp();
      int rank = 0;
#pragma unroll 1
      for (int j = 0; j < longest; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&sm.key[q][j]);
        const int4 oe = *reinterpret_cast<const int4*>(&sm.e[q][j]);
        rank += o.x > key || (o.x == key && oe.x < e);
        rank += o.y > key || (o.y == key && oe.y < e);
        rank += o.z > key || (o.z == key && oe.z < e);
        rank += o.w > key || (o.w == key && oe.w < e);
      }
      if (c < n && rank < r.K) {
        sm.out_s[q][rank] = score;
        sm.out_e[q][rank] = e;
      }
      __syncwarp();
      const bool slot = n > 0 && c < r.K;
      float s = slot ? sm.out_s[q][c] : 0.0f;
      if (r.renormalize) {
        float sum = s;
        if (!paired) sum += __shfl_xor_sync(all, sum, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(all, sum, o);
        s = s / (sum + SELECT_SUM_EPS);
      }
      if (slot) {
        ids[q * r.K + c] = sm.out_e[q][c];
        w[q * r.K + c] = s * r.scale;
      }
    }
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
