// adapter_outer.cuh - the gradients of an adapter's factors: sums over its rows of
// hidden[row] (as a column) times x[row] (as a row).
//
// Each row of x is read once for all ranks.  A CTA takes up to `unit` rows of one
// adapter and 512 columns, 64 a warp; the contraction runs across rows, with x
// straight from memory into fragments (adapter_common.cuh) and hidden as two
// 16-bit parts through shared memory, 64 rows at a time.  The CTAs' FP32 sums
// are joined by a second kernel in the order of the rows.
#pragma once

#include "adapter_common.cuh"

namespace moe {

constexpr int OUTER_STAGE = 64;                     // rows whose hidden is staged together
constexpr int OUTER_COLUMNS = ADAPTER_WARPS * 64;   // of a CTA

// MT: groups of 16 ranks.
template <typename T, int MT, bool VEC>
__global__ void __launch_bounds__(ADAPTER_THREADS) adapter_outer_kernel(const OuterArgs a) {
  constexpr int KS = OUTER_STAGE / 16;
  constexpr bool SCALED = !std::is_same<T, __nv_bfloat16>::value;
  __shared__ uint4 frags[2][KS * MT * 2 * 32];
  __shared__ Piece found;
  __shared__ float warp_max[2][ADAPTER_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  const Piece p = find_piece(a.starts, a.L, a.unit, blockIdx.x, &found);
  if (p.group < 0) return;
  const int side = blockIdx.y < a.blocks[0] ? 0 : 1;  // down's gradient, then up's
  const int n0 = (blockIdx.y - (side ? a.blocks[0] : 0)) * OUTER_COLUMNS + warp * 64;
  const int N = a.width[side], rank0 = blockIdx.z * MT * 16;
  const T* x = static_cast<const T*>(a.x[side]);
  const int64_t stride = a.stride[side];
  const float* hidden = a.hidden[side];
  const int32_t* rows = a.row_list + p.start;

  // Fragments of hidden rows at .. at+63 into buffer b; with FP16, scaled by
  // 2^-e, e the largest exponent so far.
  int top = 1;  // biased exponent of the scale in use
  float rescale = 1.0f;
  const auto stage = [&](int at, int b) {
    constexpr int WORK = KS * MT;  // a warp's lanes fill one of them
    float v[(WORK + ADAPTER_WARPS - 1) / ADAPTER_WARPS][8];
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < (WORK + ADAPTER_WARPS - 1) / ADAPTER_WARPS; ++w) {
      const int i = warp + w * ADAPTER_WARPS, ks = i / MT, mt = i % MT;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        // q: [second eight rows of 16][second eight ranks][odd row]
        const int r = at + 16 * ks + 2 * t + (q & 1) + 8 * (q >> 2), c = rank0 + 16 * mt + g + 8 * ((q >> 1) & 1);
        v[w][q] = i < WORK && r < p.count && c < a.rank ? hidden[(int64_t)rows[r] * a.rank + c] : 0.0f;
        m = fmaxf(m, fabsf(v[w][q]));
      }
    }
    float s = 1.0f;
    if constexpr (SCALED) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) warp_max[b][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < ADAPTER_WARPS; ++w) m = fmaxf(m, warp_max[b][w]);
      const int e = min((int)(__float_as_uint(m) >> 23), 253);  // (infinities stay infinite)
      const int was = top;
      top = max(top, e);
      s = __uint_as_float((uint32_t)(254 - top) << 23);
      // (sums so far are of the old scale: 2^(was - top) of it)
      rescale = top - was >= 126 ? 0.0f : __uint_as_float((uint32_t)(127 + was - top) << 23);
    }
#pragma unroll
    for (int w = 0; w < (WORK + ADAPTER_WARPS - 1) / ADAPTER_WARPS; ++w) {
      const int i = warp + w * ADAPTER_WARPS;
      if (i < WORK) {
        uint4 hi, lo;
        split2<T>(v[w][0] * s, v[w][1] * s, hi.x, lo.x);
        split2<T>(v[w][2] * s, v[w][3] * s, hi.y, lo.y);
        split2<T>(v[w][4] * s, v[w][5] * s, hi.z, lo.z);
        split2<T>(v[w][6] * s, v[w][7] * s, hi.w, lo.w);
        frags[b][(i * 2) * 32 + lane] = hi;
        frags[b][(i * 2 + 1) * 32 + lane] = lo;
      }
    }
  };

  float d[MT][8][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[m][j][i] = 0.0f;

  for (int at = 0, b = 0; at < p.count; at += OUTER_STAGE, b ^= 1) {
    stage(at, b);
    __syncthreads();
    if constexpr (SCALED) {
      if (rescale != 1.0f) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[m][j][i] *= rescale;
      }
    }
    if (n0 >= N) continue;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = at + 16 * ks + 2 * t + (i & 1) + 8 * (i >> 1);
        const bool on = r < p.count;
        q[i] = load8<T, VEC>(x + (on ? rows[r] : 0) * stride, n0 + 8 * g, N, on);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 hi = frags[b][((ks * MT + m) * 2) * 32 + lane], lo = frags[b][((ks * MT + m) * 2 + 1) * 32 + lane];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b0 = pair_of(q[0], q[1], j), b1 = pair_of(q[2], q[3], j);
          mma16816(d[m][j], hi, b0, b1, T());
          mma16816(d[m][j], lo, b0, b1, T());
        }
      }
    }
  }
  if (n0 >= N) return;
  const float back = SCALED ? __uint_as_float((uint32_t)top << 23) : 1.0f;
  float* sums = a.sums[side] + (int64_t)blockIdx.x * a.rank * N;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      // rank row g or g + 8, columns n0 + 16t + 0..7 or 8..15
      const int c = rank0 + 16 * m + g + 8 * (h >> 1), col = n0 + 16 * t + 8 * (h & 1);
      if (c >= a.rank) continue;
      float* o = sums + (int64_t)c * N;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < N) o[col + j] = d[m][j][h] * back;
    }
}

// A factor's gradient: its pieces' sums in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) adapter_join_kernel(const OuterArgs a) {
  pdl_wait();
  const int side = blockIdx.z, group = blockIdx.y;
  const int64_t n = (int64_t)a.rank * a.width[side];
  const int lo = a.starts[group], hi = a.starts[group + 1];
  const int parts = (hi - lo + a.unit - 1) / a.unit;
  if (a.alone && parts == 1) return;  // (written already)
  const float* sums = a.sums[side] + (lo / a.unit + group) * n;
  T* out = static_cast<T*>(a.grad[side]) + group * n;
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += sums[p * n + i];
    out[i] = from_f32<T>(s);
  }
}

template <typename T>
cudaError_t launch_join(const OuterArgs& a, cudaStream_t s) {
  const int64_t n = (int64_t)a.rank * std::max(a.width[0], a.width[1]);
  const dim3 grid((unsigned)std::min<int64_t>((n + 255) / 256, 1024), (unsigned)a.L, 2);
  return launch_k(adapter_join_kernel<T>, grid, dim3(256), 0, s, true, a);
}

template <typename T, int MT>
cudaError_t launch_outer_mt(const OuterArgs& a, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)pieces_of(a.rows, a.L, a.unit), (unsigned)(a.blocks[0] + a.blocks[1]),
                  (unsigned)((a.rank + 16 * MT - 1) / (16 * MT)));
  return launch_k(vec ? adapter_outer_kernel<T, MT, true> : adapter_outer_kernel<T, MT, false>, grid,
                  dim3(ADAPTER_THREADS), 0, s, true, a);
}

template <typename T>
cudaError_t launch_outer(const OuterArgs& a, bool vec, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const int mt = (a.rank + 15) / 16;
  if (mt == 1)
    e = launch_outer_mt<T, 1>(a, vec, s);
  else if (mt == 2)
    e = launch_outer_mt<T, 2>(a, vec, s);
  else if (mt == 3)
    e = launch_outer_mt<T, 3>(a, vec, s);
  else
    e = launch_outer_mt<T, 4>(a, vec, s);
  return e == cudaSuccess ? launch_join<T>(a, s) : e;
}

}  // namespace moe
