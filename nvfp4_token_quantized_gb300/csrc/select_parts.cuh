// select_parts.cuh - the choice of experts of large batches: P threads a row.
//
// A warp per row (route_select.cuh) has the least latency, but each of its K
// rounds takes a maximum over the warp and touches every lane, some 500 issue
// slots a row, and issue slots are what bounds it.  Here (131072 x 256 FP32
// sigmoid scores with a bias, 4 of 8 groups, top-8: 69 us for 143 MB, of which
// the bytes take 21; loads and trees 29, scores 4, groups 12, rounds 15, the
// slots' scores and weights 9) a warp takes 32 / P
// rows: their logits pass through registers once, a lane a column (loads, and
// of a biased sigmoid the scores), into shared memory; then each thread owns
// 32 R columns of one row and keeps their maxima in a tree: R of them in
// registers, four below each, eight columns below each of those.  A round
// compares R + 4 + 8 values instead of the whole row's, for all of the warp's
// rows at once.  Columns already chosen, and those past the last expert, are
// NaN, which no maximum takes and no comparison finds; closed ones and those
// of groups left out are -inf, so that rows with too few open experts need no
// path of their own.
#pragma once

#include "route_select.cuh"

namespace moe {

template <int R, int P>
struct PartLayout {
  static constexpr int ROWS = 32 / P;        // of a warp
  static constexpr int COLUMNS = 32 * R;     // of a thread
  static constexpr int WIDTH = COLUMNS * P;  // of a row
  // Strides in words, odd multiples of 16 bytes: eight lanes' 16-byte
  // accesses at one column of eight rows take every bank once.
  static constexpr int ROW = WIDTH + 4;
  static constexpr int MAXIMA = R == 1 ? 4 : 4 * R + 4;
  static constexpr int GROUPS_AT = ROWS * ROW + 32 * MAXIMA;
  // per row: the groups' scores, the softmax's maximum and sum, the slots
  __host__ __device__ static int totals_at(const RouteRule& r) {
    return GROUPS_AT + (r.top_groups < r.groups ? ROWS * (r.groups | 1) : 0);
  }
  __host__ __device__ static int slots_at(const RouteRule& r) { return totals_at(r) + 2 * ROWS; }
  __host__ __device__ static int words(const RouteRule& r) { return (slots_at(r) + (ROWS * r.K + 1) / 2 + 3) & ~3; }
};

__device__ __forceinline__ float max_of(float4 a) { return fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)); }
// The first place of m in a, or 0.
__device__ __forceinline__ int first_of(float4 a, float m) { return a.x == m ? 0 : a.y == m ? 1 : a.z == m ? 2 : 3; }

constexpr int CLOSED_SLOT = 0x8000;

// A lane's columns of a row: chunks of four, or every 32nd; NaN past the last.
template <typename T, int NE>
__device__ __forceinline__ void load_columns(const T* row, int E, bool vec, int lane, float (&v)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) v[i] = __int_as_float(0x7fffffff);
  if (vec) {
#pragma unroll
    for (int c = 0; c < NE; c += 4) {
      const int e = (c * 8 + lane) * 4;
      if (e >= E) continue;
      if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4*>(row + e);
        v[c] = f.x, v[c + 1] = f.y, v[c + 2] = f.z, v[c + 3] = f.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(row + e);
        const float2 a = unpack2(q.x, T()), b = unpack2(q.y, T());
        v[c] = a.x, v[c + 1] = a.y, v[c + 2] = b.x, v[c + 3] = b.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i * 32 + lane < E) v[i] = to_f32(row[i * 32 + lane]);
  }
}

// One warp a CTA (four were 3 % slower).  r.vec: whole chunks of four logits
// may be loaded.
template <int R, int P>
__global__ void __launch_bounds__(32)
    select_parts_kernel(const RouteRule r, const void* __restrict__ logits, int dtype, int64_t stride,
                        const float* __restrict__ bias, int64_t rows, int32_t* __restrict__ ids,
                        float* __restrict__ w) {
  using L = PartLayout<R, P>;
  constexpr int NE = R * P < 4 ? 4 : R * P, ROWS = L::ROWS;
  constexpr int BATCH = 32 / NE;  // rows whose loads are in flight together
  constexpr unsigned all = 0xffffffffu;
  const float none = __int_as_float(0x7fffffff);
  extern __shared__ float4 shared[];
  const int lane = threadIdx.x;
  float* buf = reinterpret_cast<float*>(shared);
  float* totals = buf + L::totals_at(r);
  uint16_t* slot = reinterpret_cast<uint16_t*>(buf + L::slots_at(r));
  const int64_t t0 = (int64_t)blockIdx.x * ROWS;
  pdl_trigger();
  pdl_wait();
  if (t0 >= rows) return;
  const int valid = rows - t0 < ROWS ? (int)(rows - t0) : ROWS;
  const bool limited = r.top_groups < r.groups;
  const bool biased_sigmoid = r.sigmoid && r.by_score;

  // The rows, a lane a column.
  float b[NE];
  bool bias_finite = true;
  if (r.by_score) {
    RouteRule flat = r;
    flat.groups = 1, flat.size = r.E, flat.lane_shift = 5;
    bias_finite = load_bias<NE>(flat, bias, lane, b);
  }
  unsigned undefined = 0;  // bit of each row without weights
  const int64_t row_bytes = stride * (dtype == MOE_DTYPE_F32 ? 4 : 2);
  const char* from = static_cast<const char*>(logits) + t0 * row_bytes;
#pragma unroll 1
  for (int q0 = 0; q0 < valid; q0 += BATCH, from += BATCH * row_bytes) {
    float v[BATCH][NE];
    auto load = [&](auto type) {
      using T = decltype(type);
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        load_columns<T, NE>(reinterpret_cast<const T*>(q0 + u < valid ? from + u * row_bytes : from), r.E, r.vec, lane,
                            v[u]);
    };
    if (dtype == MOE_DTYPE_F32) load(float());
    else if (dtype == MOE_DTYPE_F16) load(__half());
    else load(__nv_bfloat16());
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int q = q0 + u;
      if (q >= valid) break;
      float sum = 0.0f;  // finite: so is every logit
      if (r.vec) {
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
          const float2 t = add2(make_float2(v[u][i], v[u][i + 1]), make_float2(v[u][i + 2], v[u][i + 3]));
          sum += (i * 8 + lane) * 4 < r.E ? t.x + t.y : 0.0f;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) sum += i * 32 + lane < r.E ? v[u][i] : 0.0f;
      }
      const bool special = __any_sync(all, !(fabsf(sum) < INFINITY));
      if (special) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int e = r.vec ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane;
          bad |= e < r.E && (v[u][i] != v[u][i] || (!r.sigmoid && v[u][i] == INFINITY));
        }
        if (__any_sync(all, bad)) undefined |= 1u << q;
      }
      if (biased_sigmoid) {
        if (special || !bias_finite) {
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            const float x = v[u][i], s = sigmoid_fast(x) + b[i];
            v[u][i] = x != x ? x : x > -INFINITY && s > -INFINITY ? s : -INFINITY;
          }
        } else {
#pragma unroll
          for (int i = 0; i < NE; ++i) v[u][i] = sigmoid_fast(v[u][i]) + b[i];
        }
      }
      float* to = buf + q * L::ROW;
      if (r.vec) {
#pragma unroll
        for (int c = 0; c < NE; c += 4) {
          const int e = (c * 8 + lane) * 4;
          if (e < L::WIDTH)
            *reinterpret_cast<float4*>(to + e) = make_float4(v[u][c], v[u][c + 1], v[u][c + 2], v[u][c + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < R * P; ++i) to[i * 32 + lane] = v[u][i];
      }
    }
  }
  __syncwarp();

  // From here on a thread has columns first .. first + COLUMNS of one row
  // (rows past the last hold what was there; nothing of them leaves).
  const int row = lane & (ROWS - 1), part = lane / ROWS, first = part * L::COLUMNS;
  float* whole_row = buf + row * L::ROW;
  float* mine = whole_row + first;
  const bool need_total = !r.sigmoid && (r.by_score || !r.renormalize);
  const bool need_top = !r.sigmoid && (need_total || (limited && r.top2));
  float top = 0.0f, total = 1.0f;
  if (need_top) {
    float m = none;
#pragma unroll
    for (int i = 0; i < L::COLUMNS; i += 4) m = fmaxf(m, max_of(*reinterpret_cast<const float4*>(mine + i)));
#pragma unroll
    for (int o = ROWS; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(all, m, o));
    top = m == -INFINITY ? 0.0f : m;
  }
  if (need_total) {
    // (NaN and -inf add nothing)
    auto power = [&](float x) { return exp_fast(fmaxf(x - top, -200.0f)); };
    OrderFree sum;
#pragma unroll 4
    for (int i = 0; i < L::COLUMNS; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(mine + i);
      sum.add(make_float2(power(x.x), power(x.y)));
      sum.add(make_float2(power(x.z), power(x.w)));
    }
    float2 t = make_float2(sum.high.x + sum.high.y, sum.low.x + sum.low.y);
#pragma unroll
    for (int o = ROWS; o < 32; o <<= 1)
      t = add2(t, make_float2(__shfl_xor_sync(all, t.x, o), __shfl_xor_sync(all, t.y, o)));
    total = t.x + t.y;
    if (total == 0.0f) total = 1.0f;
    if (r.by_score) {
      const float k = 1.0f / total;
#pragma unroll 4
      for (int i = 0; i < L::COLUMNS; ++i) {
        if (first + i >= r.E) break;
        const float x = mine[i];
        float s = fmaf(exp_fast(x - top), k, __ldg(bias + first + i));
        if (x == -INFINITY || (!bias_finite && !(s > -INFINITY))) s = -INFINITY;
        mine[i] = s;
      }
    }
  }
  if (limited) {
    // The groups' scores, a thread every P-th group, then their ranks; the
    // columns of the groups left out close.
    float* scores = buf + L::GROUPS_AT + row * (r.groups | 1);
    __syncwarp();
    for (int g = part; g < r.groups; g += P) {
      const float* x = whole_row + g * r.size;
      float b1 = -INFINITY, b2 = -INFINITY;
      if (!r.top2) {
        if (r.size % 4 == 0) {
#pragma unroll 4
          for (int i = 0; i < r.size; i += 4) b1 = fmaxf(b1, max_of(*reinterpret_cast<const float4*>(x + i)));
        } else {
#pragma unroll 4
          for (int i = 0; i < r.size; ++i) b1 = fmaxf(b1, x[i]);
        }
      } else {
        if (r.size % 4 == 0) {
#pragma unroll 4
          for (int i = 0; i < r.size; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(x + i);
            const float c1 = fmaxf(f.x, f.y), d1 = fmaxf(f.z, f.w);
            const float c2 = fmaxf(fmaxf(fminf(f.x, f.y), fminf(f.z, f.w)), fminf(c1, d1));
            merge2(b1, b2, fmaxf(c1, d1), c2);
          }
        } else {
#pragma unroll 4
          for (int i = 0; i < r.size; ++i) {
            b2 = fmaxf(b2, fminf(b1, x[i]));
            b1 = fmaxf(b1, x[i]);
          }
        }
        if (b1 > -INFINITY) {
          // (of a softmax, what its sum would divide)
          if (!r.by_score) {
            b1 = r.sigmoid ? sigmoid_fast(b1) : exp_fast(b1 - top);
            b2 = r.sigmoid ? sigmoid_fast(b2) : exp_fast(b2 - top);
          }
          if (b2 > -INFINITY) b1 += b2;
        }
      }
      scores[g] = b1;
    }
    __syncwarp();
    for (int g = part; g < r.groups; g += P) {
      const float s = scores[g];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < r.groups; ++j) {
        const float o = scores[j];
        rank += j < g ? o >= s : o > s;
      }
      if (rank < r.top_groups) continue;
      float* x = whole_row + g * r.size;
      if (r.size % 4 == 0) {
        for (int i = 0; i < r.size; i += 4)
          *reinterpret_cast<float4*>(x + i) = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      } else {
        for (int i = 0; i < r.size; ++i) x[i] = -INFINITY;
      }
    }
    __syncwarp();
  }

  // The tree, and K rounds.
  auto eight = [&](const float* x) {
    const float4* f = reinterpret_cast<const float4*>(x);
    return fmaxf(max_of(f[0]), max_of(f[1]));
  };
  float4* maxima = reinterpret_cast<float4*>(buf + ROWS * L::ROW + lane * L::MAXIMA);
  float best[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float4 m = make_float4(eight(mine + i * 32), eight(mine + i * 32 + 8), eight(mine + i * 32 + 16),
                                 eight(mine + i * 32 + 24));
    maxima[i] = m;
    best[i] = max_of(m);
  }
  unsigned before = 0;  // the lanes of the row's lower parts
#pragma unroll
  for (int p = 0; p < P; ++p) before |= p < part ? 1u << (row + p * ROWS) : 0u;
#pragma unroll 1
  for (int k = 0; k < r.K; ++k) {
    float m = best[0];
#pragma unroll
    for (int i = 1; i < R; ++i) m = fmaxf(m, best[i]);
    float most = m;
    bool wins = true;
    if constexpr (P > 1) {
#pragma unroll
      for (int o = ROWS; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(all, most, o));
      wins = m == most;
      const unsigned others = __ballot_sync(all, wins);
      wins = wins && !(others & before);
    }
    if (k == 0 && !need_top) top = most == -INFINITY ? 0.0f : most;
    if (wins) {
      int i = 0;
#pragma unroll
      for (int u = R - 1; u > 0; --u) i = best[u] == m ? u : i;
      if (best[0] == m) i = 0;
      const int j = first_of(maxima[i], m);
      float* leaf = mine + i * 32 + j * 8;
      const float4 low = reinterpret_cast<const float4*>(leaf)[0], high = reinterpret_cast<const float4*>(leaf)[1];
      const int at = max_of(low) == m ? first_of(low, m) : 4 + first_of(high, m);
      slot[row * r.K + k] = (uint16_t)((first + i * 32 + j * 8 + at) | (m == -INFINITY ? CLOSED_SLOT : 0));
      leaf[at] = none;
      reinterpret_cast<float*>(maxima + i)[j] = eight(leaf);
      const float now = max_of(maxima[i]);
#pragma unroll
      for (int u = 0; u < R; ++u) best[u] = u == i ? now : best[u];
    }
  }
  if (part == 0) {
    totals[row] = top;
    totals[ROWS + row] = total;
  }
  __syncwarp();

  // The slots of several rows at a time, a lane each.
  const int slots = 1 << r.slot_shift, at_once = 32 >> r.slot_shift;
#pragma unroll 1
  for (int q0 = 0; q0 < valid; q0 += at_once) {
    const int q = q0 + (lane >> r.slot_shift), c = lane & (slots - 1);
    const bool has = q < valid && c < r.K;
    const bool lost = has && (undefined >> q & 1);  // (whose slots may not have been written)
    float s = 0.0f;
    int e = 0;
    if (has && !lost) {
      const int x = slot[q * r.K + c];
      e = x & (CLOSED_SLOT - 1);
      if (!(x & CLOSED_SLOT)) {
        const float l = logit_at(row_at(logits, dtype, (t0 + q) * stride), dtype, e);
        s = r.sigmoid ? sigmoid_ieee(l) : expf(l - totals[q]) / totals[ROWS + q];
      }
    }
    if (r.renormalize) {
      float sum = s;
#pragma unroll 1
      for (int o = slots >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(all, sum, o);
      s = s / (sum + SELECT_SUM_EPS);
    }
    if (has) {
      ids[(t0 + q) * r.K + c] = lost ? c : e;
      w[(t0 + q) * r.K + c] = lost ? none : s * r.scale;
    }
  }
}

}  // namespace moe
