// adapter_apply.cuh - rows through their adapters, a few hundred at most (a decode
// step's):
// hidden = scale x down^T, out = base + hidden up, in one launch.
//
// Bound by the adapters' bytes and by latency.  A cluster takes up to 32 rows of one
// adapter, which its CTAs find in ids themselves (more rows a tile would read the
// factors less often, but leave CTAs idle: 128 rows of one adapter, rank 64, 4096
// wide, 20 us, in one tile of 128 rows 46); the CTAs split the first
// product's long axis, add their parts through distributed shared memory, and
// split the second product's columns, so that few rows still spread over the GPU.
// Within a CTA a warp has 16 rows; fewer rows leave more warps for the split.  The
// operands go from memory into the fragments of mma.sync (adapter_common.cuh): with
// one to some rows an adapter a tile of 128 would be empty for the most part.  64
// rows on 16 adapters, rank 16, 2048 to 2048: 5.8 us a call in a replayed graph, a
// chain of latencies (launch, ids, rows, two exchanges, rows).
//
// hidden is FP32; the second product takes it as two 16-bit parts (split2), as a
// single rounding would show beside the output's own.
#pragma once

#include <cooperative_groups.h>

#include "adapter_common.cuh"

namespace moe {
namespace cg = cooperative_groups;

template <int NT>
struct ApplyShared {
  static constexpr int R = 8 * NT, RP = hidden_pitch(R), KS = (NT + 1) / 2;
  static constexpr int PART = ADAPTER_WARPS * 16 * RP * 4;                  // sums, then fragments
  static constexpr int FRAGS = (APPLY_TILE / 16) * KS * 2 * 512;
  static constexpr int FIRST = PART > FRAGS ? PART : FRAGS;
  static constexpr int BYTES = FIRST + APPLY_TILE * RP * 4;
};

template <typename T, int NT, bool VEC>
__global__ void __launch_bounds__(ADAPTER_THREADS, NT <= 8 ? 2 : 1) adapter_apply_kernel(const AdapterArgs a) {
  using S = ApplyShared<NT>;
  constexpr int R = S::R, RP = S::RP, KS = S::KS;
  extern __shared__ __align__(16) unsigned char smem[];
  float* part = reinterpret_cast<float*>(smem);
  uint4* frags = reinterpret_cast<uint4*>(smem);
  float* hid = reinterpret_cast<float*>(smem + S::FIRST);
  __shared__ int row_of[APPLY_TILE];
  __shared__ int counts[FEW_ROWS / 32], place;  // the group's rows among 32 each; of row `number`
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int C = a.cluster, crank = blockIdx.x % C, number = blockIdx.x / C;

  // ---- the group's rows, found in ids ----
  // A cluster stands for a tile that an adapter's rows may fill, or, where there are
  // more of those than rows, for a row, and takes a tile if that row is its first.
  const bool by_row = a.tiles == a.rows;
  const int group = by_row ? adapter_key(a.ids[number], a.L) : number / a.subs;
  constexpr int PASSES = FEW_ROWS / ADAPTER_THREADS;
  int at[PASSES];  // places of this thread's rows among the group's, -1: another's
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = tid + i * ADAPTER_THREADS;
    const bool mine = row < a.rows && adapter_key(a.ids[row], a.L) == group;
    const unsigned m = __ballot_sync(0xffffffffu, mine);
    at[i] = mine ? __popc(m & ((1u << lane) - 1)) : -1;
    if (lane == 0) counts[warp + i * ADAPTER_WARPS] = __popc(m);
  }
  __syncthreads();
  const int n = lane < FEW_ROWS / 32 ? counts[lane] : 0, total = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int before = __reduce_add_sync(0xffffffffu, lane < warp + i * ADAPTER_WARPS ? n : 0);
    if (at[i] >= 0) at[i] += before;
    if (by_row && tid + i * ADAPTER_THREADS == number) place = at[i];
  }
  if (total == 0) return;  // (the whole cluster)
  __syncthreads();
  const int begin = by_row ? place : number % a.subs * APPLY_TILE, count = min(APPLY_TILE, total - begin);
  if (count <= 0 || begin % APPLY_TILE != 0) return;
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    if (at[i] >= begin && at[i] < begin + count) row_of[at[i] - begin] = tid + i * ADAPTER_THREADS;
  __syncthreads();

  const T* x = static_cast<const T*>(a.x);
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.out);
  const int K = a.in, N = a.n_out;

  if (group == a.L) {
    rows_without_adapter<T, VEC>(a, row_of, count, crank, C);
    return;
  }

  // warps: wm groups of 16 rows, the rest splits the long axes
  const int wm = count <= 16 ? 1 : 2;
  const int ways = ADAPTER_WARPS / wm, rg = warp & (wm - 1), way = warp / wm;
  const int r0 = rg * 16 + g, r1 = r0 + 8;
  const bool on0 = r0 < count, on1 = r1 < count;
  const int64_t row0 = on0 ? row_of[r0] : 0, row1 = on1 ? row_of[r1] : 0;

  // ---- hidden: this warp's 16 rows, its share of the long axis ----
  {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    const int units = (K + 31) / 32, slices = C * ways;
    const int per = (units + slices - 1) / slices;
    const int u0 = (crank * ways + way) * per, u1 = min(units, u0 + per);
    if (rg * 16 < count) {
      const T* x0 = x + row0 * a.x_stride;
      const T* x1 = x + row1 * a.x_stride;
      const T* w = static_cast<const T*>(a.first) + (int64_t)group * a.rank * K;
      constexpr int U = NT <= 2 ? 4 : NT <= 8 ? 2 : 1;  // units in flight
      for (int u = u0; u < u1; u += U) {
        uint4 q0[U], q1[U], b[U][NT];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int col = (u + i) * 32 + t * 8;
          const bool in = u + i < u1;
          q0[i] = load8<T, VEC>(x0, col, K, in && on0);
          q1[i] = load8<T, VEC>(x1, col, K, in && on1);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            b[i][j] = load8<T, VEC>(w + (int64_t)(8 * j + g) * K, col, K, in && 8 * j + g < a.rank);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint4 first = make_uint4(q0[i].x, q1[i].x, q0[i].y, q1[i].y);
          const uint4 second = make_uint4(q0[i].z, q1[i].z, q0[i].w, q1[i].w);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16816(acc[j], first, b[i][j].x, b[i][j].y, T());
            mma16816(acc[j], second, b[i][j].z, b[i][j].w, T());
          }
        }
      }
    }
    // part[way][row][rank]
    float* p0 = part + ((way * wm + rg) * 16 + g) * RP + 2 * t;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(p0 + 8 * j) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(p0 + 8 * RP + 8 * j) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  // ---- its parts added: the CTA's ways, then the cluster's CTAs ----
  const float scale = a.scales ? a.scales[group] : 1.0f;
  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) {
    if (ways > 1) {
      for (int i = tid; i < count * R; i += ADAPTER_THREADS) {
        float* p = part + (i / R) * RP + i % R;
        float s = *p;
        for (int w = 1; w < ways; ++w) s += p[w * wm * 16 * RP];
        *p = s;
      }
    }
    cluster.sync();
  }
  for (int i = crank * ADAPTER_THREADS + tid; i < count * R; i += C * ADAPTER_THREADS) {
    const int r = i / R, c = i % R, at = r * RP + c;
    float s = 0.0f;
    if (C > 1) {
      for (int p = 0; p < C; ++p) s += cluster.map_shared_rank(part, (crank + p) % C)[at];  // (each begins at its own)
    } else {
      for (int w = 0; w < ways; ++w) s += part[w * wm * 16 * RP + at];
    }
    s = c < a.rank ? s * scale : 0.0f;  // (nothing for the ranks that fill up)
    if (a.hidden && c < a.rank) a.hidden[(int64_t)row_of[r] * a.rank + c] = s;
    if (C > 1) {
      for (int p = 0; p < C; ++p) cluster.map_shared_rank(hid, (crank + p) % C)[at] = s;
    } else {
      hid[at] = s;
    }
  }
  if (C > 1)
    cluster.sync();  // (the last access to another CTA's shared memory lies before)
  else
    __syncthreads();

  // ---- hidden as fragments, two parts each ----
  float back0 = 1.0f, back1 = 1.0f;
  {
    const float* h0 = hid + r0 * RP + 2 * t;
    const float* h1 = h0 + 8 * RP;
    float s0 = 1.0f, s1 = 1.0f;
    if constexpr (sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value) {
      float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (on0) m0 = fmaxf(m0, fmaxf(fabsf(h0[8 * j]), fabsf(h0[8 * j + 1])));
        if (on1) m1 = fmaxf(m1, fmaxf(fabsf(h1[8 * j]), fabsf(h1[8 * j + 1])));
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
      }
      s0 = exponent_scale(m0, back0);
      s1 = exponent_scale(m1, back1);
    }
    for (int ks = way; ks < KS; ks += ways) {
      float v[4][2];  // row 0 and 1 at the first eight ranks, then at the second
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = 16 * ks + 8 * (q >> 1);
        const bool have = c < R && (q & 1 ? on1 : on0);
        const float2 f = have ? *reinterpret_cast<const float2*>((q & 1 ? h1 : h0) + c) : make_float2(0.0f, 0.0f);
        const float s = q & 1 ? s1 : s0;
        v[q][0] = f.x * s;
        v[q][1] = f.y * s;
      }
      uint4 hi, lo;
      split2<T>(v[0][0], v[0][1], hi.x, lo.x);
      split2<T>(v[1][0], v[1][1], hi.y, lo.y);
      split2<T>(v[2][0], v[2][1], hi.z, lo.z);
      split2<T>(v[3][0], v[3][1], hi.w, lo.w);
      frags[((rg * KS + ks) * 2) * 32 + lane] = hi;
      frags[((rg * KS + ks) * 2 + 1) * 32 + lane] = lo;
    }
  }
  __syncthreads();
  if (rg * 16 >= count) return;

  // ---- out: 64 columns at a time ----
  const T* up = static_cast<const T*>(a.second) + (int64_t)group * a.rank * N;
  for (int n0 = (crank * ways + way) * 64; n0 < N; n0 += C * ways * 64) {
    const int oc = n0 + 16 * t;
    uint4 y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      y[q] = base ? load8<T, VEC>(base + (q & 1 ? row1 : row0) * a.base_stride, oc + 8 * (q >> 1), N, q & 1 ? on1 : on0)
                  : make_uint4(0, 0, 0, 0);
    float d[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint4 b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = 16 * ks + 2 * t + (q & 1) + 8 * (q >> 1);
        b[q] = load8<T, VEC>(up + (int64_t)k * N, n0 + 8 * g, N, k < a.rank);
      }
      const uint4 hi = frags[((rg * KS + ks) * 2) * 32 + lane], lo = frags[((rg * KS + ks) * 2 + 1) * 32 + lane];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b0 = pair_of(b[0], b[1], j), b1 = pair_of(b[2], b[3], j);
        mma16816(d[j], hi, b0, b1, T());
        mma16816(d[j], lo, b0, b1, T());
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // columns oc + 8 * (q >> 1) + 0..7 of row q & 1: d[0..7][i]
      const int i = (q & 1) * 2 + (q >> 1);
      const float back = q & 1 ? back1 : back0;
      const uint32_t w[4] = {y[q].x, y[q].y, y[q].z, y[q].w};
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 f = unpack2(w[p], T());
        o[p] = pack2(fmaf(d[2 * p][i], back, f.x), fmaf(d[2 * p + 1][i], back, f.y), T());
      }
      if (q & 1 ? on1 : on0)
        store8<T, VEC>(out + (q & 1 ? row1 : row0) * a.out_stride, oc + 8 * (q >> 1), N,
                       make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

template <typename T, int NT, bool VEC>
cudaError_t launch_apply_one(const AdapterArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = adapter_apply_kernel<T, NT, VEC>;
  constexpr int bytes = ApplyShared<NT>::BYTES;
  if (bytes > 46 * 1024) {
    const cudaError_t e = raise_shared(kernel, bytes, done);
    if (e != cudaSuccess) return e;
  }
  return launch_clustered(kernel, a, ADAPTER_THREADS, bytes, false, s);
}

template <typename T>
cudaError_t launch_apply(const AdapterArgs& a, bool vec, cudaStream_t s) {
  switch ((a.rank + 7) / 8) {
#define MOE_APPLY(NT) return vec ? launch_apply_one<T, NT, true>(a, s) : launch_apply_one<T, NT, false>(a, s)
    case 1: MOE_APPLY(1);
    case 2: MOE_APPLY(2);
    case 3: MOE_APPLY(3);
    case 4: MOE_APPLY(4);
    case 5:
    case 6: MOE_APPLY(6);
    case 7:
    case 8: MOE_APPLY(8);
  }
  MOE_APPLY(16);
#undef MOE_APPLY
}

}  // namespace moe
