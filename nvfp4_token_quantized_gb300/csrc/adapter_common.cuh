// adapter_common.cuh - what the kernels of the low-rank adapters share: the
// tensor cores' 16 x 8 x 16 product on register fragments, loads of eight
// neighbouring elements, and the rows grouped by adapter.
//
// Fragments without shared memory.  A product may number its contraction and
// its columns as it likes, as long as both operands agree, so each lane loads
// 16 bytes of a row and hands them out to the fragments in the order it has:
//  - contraction along the rows' long axis (hidden = x down^T): of 32 elements a
//    lane (quad position t) holds 8t .. 8t+7; elements 0..3 are its four of the
//    first product, 4..7 those of the second, in both operands;
//  - contraction across rows (out = hidden up, gradients): a lane loads columns
//    8g .. 8g+7 (g = lane / 4) of rows 2t, 2t+1, 2t+8, 2t+9; product j of eight
//    takes column 8g + j from it, so the eight accumulators of a lane hold 16
//    neighbouring columns, which are moved by two 16-byte accesses a row.
#pragma once

#include "common.cuh"
#include "elem_types.cuh"
#include "kernels_ops.h"

#include <type_traits>

namespace moe {

constexpr int ADAPTER_THREADS = 256;
constexpr int ADAPTER_WARPS = ADAPTER_THREADS / 32;
constexpr int ADAPTER_TILE = 128;  // rows of a tile: 16 a warp
constexpr int FEW_ROWS = 512;      // most rows of a forward in one launch
constexpr int APPLY_TILE = 32;     // rows of its clusters
constexpr int GRADIENT_ROWS = 32;  // rows of a stage of the factors' gradients

__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Elements col .. col+7 of a row, zeros from `width` on and where !on.  VEC:
// rows start on 16 bytes and width is a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load8(const T* row, int col, int width, bool on) {
  uint4 q = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    if (on && col < width) q = *reinterpret_cast<const uint4*>(row + col);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + col;
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = on && col + i < width ? p[i] : 0u;
    q = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  return q;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int col, int width, const uint4& q) {
  if constexpr (VEC) {
    if (col < width) *reinterpret_cast<uint4*>(row + col) = q;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// Element j of two rows' eight, packed (the first row's in the low half).
__device__ __forceinline__ uint32_t pair_of(const uint4& a, const uint4& b, int j) {
  const uint32_t wa = j < 2 ? a.x : j < 4 ? a.y : j < 6 ? a.z : a.w;
  const uint32_t wb = j < 2 ? b.x : j < 4 ? b.y : j < 6 ? b.z : b.w;
  return __byte_perm(wa, wb, j & 1 ? 0x7632 : 0x5410);
}

// Two FP32 values as T plus what T leaves of them, as T: hi + lo keeps 16 bits
// and more (22 for FP16 near 1), so a product with both loses nothing that the
// output's own rounding would show.
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b, T());
  const float2 h = unpack2(hi, T());
  lo = pack2(isinf(h.x) ? 0.0f : a - h.x, isinf(h.y) ? 0.0f : b - h.y, T());
}

// The power of two that brings values up to m in size to 2^14 .. 2^15, and (back) its
// inverse: FP16 parts of scaled values do not overflow, and split2's, whose last bit
// is 2^-24 at least, keep 16 bits down to 2^-22 of m and to 2^-39 of m what is
// smaller.  (Products and sums are FP32: 2^15 leaves room for any 16-bit factor.)
// Both are normal numbers; an infinite m counts as the largest finite one.
__device__ __forceinline__ float exponent_scale(float m, float& back) {
  const int e = min((int)(__float_as_uint(m) >> 23), 254);  // m >= 0
  const int b = min(127 + 14 - (e - 127), 253);             // (at least 14)
  back = __uint_as_float((uint32_t)(254 - b) << 23);
  return __uint_as_float((uint32_t)b << 23);
}

// ---- rows by adapter ----

// Group i's rows are rows[starts[i]] .. rows[starts[i + 1] - 1], in ascending
// order.  Of few adapters every one is a group, and L the rows without one; of many
// only those that have rows, in ascending order (group_of says which; groups behind
// the last begin at T).
__device__ __forceinline__ int adapter_key(int id, int L) { return (unsigned)id < (unsigned)L ? id : L; }

// Row pitch of FP32 tiles in shared memory: the eight rows and four pairs of a
// fragment fall into different banks.
__host__ __device__ constexpr int hidden_pitch(int R) { return R + (40 - R % 32) % 32; }

// A tile of rows without an adapter: base alone, by the C CTAs of a cluster.
template <typename T, bool VEC>
__device__ __forceinline__ void rows_without_adapter(const AdapterArgs& a, const int* row_of, int count, int crank,
                                                     int C) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.out);
  for (int r = crank * ADAPTER_WARPS + warp; r < count; r += C * ADAPTER_WARPS) {
    const int64_t row = row_of[r];
    if (a.hidden)
      for (int i = lane; i < a.rank; i += 32) a.hidden[row * a.rank + i] = 0.0f;
    if (out == base) continue;
    constexpr int U = 8;  // accesses in flight: one at a time the row takes a latency each
    for (int c = lane * 8; c < a.n_out; c += 256 * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = load8<T, VEC>(base + row * a.base_stride, c + 256 * u, a.n_out, base != nullptr);
#pragma unroll
      for (int u = 0; u < U; ++u) store8<T, VEC>(out + row * a.out_stride, c + 256 * u, a.n_out, v[u]);
    }
  }
}

// tiles x cluster CTAs; pdl: may start while its predecessor finishes.
template <typename K>
cudaError_t launch_clustered(K kernel, const AdapterArgs& a, int threads, int bytes, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.tiles * a.cluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)a.cluster, 1, 1};
  cfg.numAttrs = 1;
  if (pdl) {
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Pieces of `unit` rows of the groups: group i's pieces have the numbers
// starts[i] / unit + i and up; numbers between two groups' may be unused.
struct Piece {
  int group;         // -1: none of the number
  int start, count;  // in rows[]
  int number;        // of the group's pieces
};

__host__ __device__ __forceinline__ int64_t pieces_of(int64_t rows, int64_t groups, int unit) {
  return rows / unit + groups;
}

// The piece of a number, by all threads of the CTA; group -1 for an unused
// number.  `found` is shared.  (Group a's numbers lie in [a, a + rows / unit].)
__device__ __forceinline__ Piece find_piece(const int32_t* starts, int64_t rows, int groups, int unit, int number,
                                            Piece* found) {
  if (threadIdx.x == 0) found->group = -1;
  __syncthreads();
  const int last = min(number, groups - 1);
  for (int a = max(number - (int)(rows / unit), 0) + threadIdx.x; a <= last; a += blockDim.x) {
    const int lo = starts[a], hi = starts[a + 1];
    const int i = number - (lo / unit + a);
    if (i >= 0 && lo + (int64_t)i * unit < hi) {
      const int at = lo + i * unit;
      *found = {a, at, min(unit, hi - at), i};
    }
  }
  __syncthreads();
  return *found;
}

}  // namespace moe
