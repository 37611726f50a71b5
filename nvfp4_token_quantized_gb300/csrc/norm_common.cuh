// norm_common.cuh - what the block norms' kernels and their gradient's share:
// the sizes of a call, the sums over a row's threads, and the ring that
// brings rows ahead of the arithmetic.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "elem_types.cuh"
#include "kernels_ops.h"

namespace moe {

// 1 / sqrt(v), v > 0: the hardware's approximation (2 units in the last
// place) and one Newton step, about one unit, without the call and the
// branches of an IEEE root and quotient that every warp of a row would make.
// 0 for a sum of squares past FP32, as 1 / sqrt gives (the step would make it
// 0 times infinity).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float y = rsqrtf(v);
  return v < INFINITY ? fmaf(0.5f * y, fmaf(-v * y, y, 1.0f), y) : y;
}

struct NormShape {
  int H;
  int lanes;  // threads of a row: a power of two up to 32, or a multiple of 32
  bool layer, branch, post, pre, gate_sigmoid, weight_f32;
  int gate;
  float eps, offset, scale, inv_h;
};

inline NormShape norm_shape(const moe_norm_config& c) {
  NormShape s{};
  s.H = c.hidden;
  s.layer = c.kind == MOE_NORM_LAYER;
  s.branch = c.branch != 0;
  s.post = c.branch && c.post;
  s.pre = c.pre != 0;
  s.gate = c.branch ? c.gate : MOE_GATE_NONE;
  s.gate_sigmoid = c.gate_sigmoid != 0;
  s.weight_f32 = c.weight_dtype == MOE_DTYPE_F32;
  s.eps = c.eps;
  s.offset = c.weight_offset;
  s.scale = c.branch_scale;
  s.inv_h = 1.0f / (float)c.hidden;
  return s;
}

// A row's threads: eight columns a thread and chunk, V chunks.  Rows of up
// to 32 threads share a warp or have one (no barrier), wider ones a CTA.
// fixed: the constant of a kernel for rows without 16-byte accesses, or 0.
inline int row_lanes(int H, int V, int fixed) {
  if (fixed) return fixed;
  const int need = (H + 8 * V - 1) / (8 * V);  // (each thread of a row of whole chunks)
  if (need > 32) return (need + 31) / 32 * 32;
  int lanes = 1;
  while (lanes < need) lanes *= 2;
  return lanes;
}
constexpr int NORM_SMALL_CTA = 128;  // threads of a CTA whose rows take a warp or less
inline int row_cta_threads(int lanes) { return lanes > 32 ? lanes : NORM_SMALL_CTA; }
inline int rows_per_cta(int lanes) { return row_cta_threads(lanes) / lanes; }

// Sums over a row's threads of N values at a time; every thread gets the same
// bits.  Inside a warp several values are summed together: each step of the
// tree hands half of them to the other half of the lanes, so four values take
// six shuffles instead of twenty.  Wider rows than a warp take one barrier:
// the warps' sums are double-buffered, so that the next sum may start while
// slow threads still read this one.  WARPS: of the largest CTA, at most 16;
// WIDE: rows are wider than a warp.
template <bool WIDE>
struct RowSums {
  static constexpr int WARPS = 16;
  // Sums of one, two and four values have places of their own, [warp][value]:
  // entries past the last warp stay 0 (clear()).
  static constexpr int HALF = (1 + 2 + 4) * WARPS;
  static constexpr int WORDS = 2 * HALF;
  float* red;  // [2][HALF]
  int lanes;  // threads of a row
  int turn = 0;
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < WORDS; i += blockDim.x) red[i] = 0.0f;
    __syncthreads();
  }
  __device__ __forceinline__ static float swap(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
  // N: 1, 2 or 4; the smaller ones' places come first
  template <int N>
  __device__ __forceinline__ float* next() {
    return red + (turn ^= 1) * HALF + (N - 1) * WARPS;
  }

  __device__ __forceinline__ void operator()(float (&v)[1]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (WIDE || o < lanes) v[0] += swap(v[0], o);
    if constexpr (!WIDE) return;
    float* buf = next<1>();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v[0];
    __syncthreads();
    // (every thread adds all partials, four at a read: half the latency of a
    // second tree, which counts where one row has the SM to itself)
    v[0] = 0.0f;
#pragma unroll
    for (int q = 0; q < WARPS / 4; ++q) {
      if (q * 128 >= lanes) break;
      const float4 f = reinterpret_cast<const float4*>(buf)[q];
      v[0] += (f.x + f.y) + (f.z + f.w);
    }
  }
  __device__ __forceinline__ void operator()(float (&v)[2]) {
    if constexpr (!WIDE) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) {
          v[0] += swap(v[0], o);
          v[1] += swap(v[1], o);
        }
      return;
    }
    const int lane = threadIdx.x & 31;
    const bool odd = lane & 1;
    // lane bit 0: which value a lane goes on with
    float mine = (odd ? v[1] : v[0]) + swap(odd ? v[0] : v[1], 1);
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) mine += swap(mine, o);
    float* buf = next<2>();
    if (lane < 2) buf[(threadIdx.x >> 5) * 2 + lane] = mine;
    __syncthreads();
    mine = buf[lane];  // warp lane / 2, value lane % 2
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) mine += swap(mine, o);
    const float other = swap(mine, 1);
    v[0] = odd ? other : mine;
    v[1] = odd ? mine : other;
  }
  __device__ __forceinline__ void operator()(float (&v)[4]) {
    if constexpr (!WIDE) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) {
#pragma unroll
          for (int n = 0; n < 4; ++n) v[n] += swap(v[n], o);
        }
      return;
    }
    const int lane = threadIdx.x & 31;
    const bool odd = lane & 1, high = lane & 2;
    // lane bit 0: values 0, 1 or 2, 3; bit 1: the first or second of them
    const float a = (odd ? v[2] : v[0]) + swap(odd ? v[0] : v[2], 1);
    const float b = (odd ? v[3] : v[1]) + swap(odd ? v[1] : v[3], 1);
    float mine = (high ? b : a) + swap(high ? a : b, 2);
#pragma unroll
    for (int o = 16; o > 2; o >>= 1) mine += swap(mine, o);
    float* buf = next<4>();
    if (lane < 4) buf[(threadIdx.x >> 5) * 4 + lane] = mine;  // value 2 (lane & 1) + (lane >> 1)
    __syncthreads();
    // lane: warps lane / 4 and 8 + lane / 4, value as above
    mine = buf[lane] + buf[32 + lane];
#pragma unroll
    for (int o = 16; o > 2; o >>= 1) mine += swap(mine, o);
    const float c = swap(mine, 2);
    const float lo = high ? c : mine, hi = high ? mine : c;
    const float lo2 = swap(lo, 1), hi2 = swap(hi, 1);
    v[0] = odd ? lo2 : lo;
    v[1] = odd ? hi2 : hi;
    v[2] = odd ? lo : lo2;
    v[3] = odd ? hi : hi2;
  }
};

// A thread's place in its row, and the columns it holds: value k of chunk v.
// VEC: rows take 16-byte accesses, a chunk is eight neighbouring columns;
// else neighbouring threads hold neighbouring columns, and the row's threads
// are a constant, LANES, so that a chunk's eight accesses differ by constants.
template <bool VEC, int LANES>
struct Place {
  int i, count;  // place; values (VEC: chunks) within the row
  int row_lanes;
  __device__ __forceinline__ Place(int place, int lanes, int H) : i(place), row_lanes(lanes) {
    const int l = this->lanes();
    count = ((VEC ? H / 8 : H) - i + l - 1) / l;
  }
  __device__ __forceinline__ int lanes() const { return VEC ? row_lanes : LANES; }
  __device__ __forceinline__ int column(int v, int k) const {
    return VEC ? (v * row_lanes + i) * 8 + k : (v * 8 + k) * LANES + i;
  }
  __device__ __forceinline__ bool in_row(int v, int k) const { return (VEC ? v : v * 8 + k) < count; }
};

// ---- rows ahead of the arithmetic ----
// VEC: a ring in shared memory filled by cp.async.  A thread copies and later
// reads only its own 16-byte pieces, so the ring needs no barrier and no flag.
// Otherwise: rows as the granules that hold them, behind a barrier (below); rows
// of more than two chunks a thread are read from global memory.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the latest N groups of copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One thread's pieces of a row of T in a ring stage: units of 16 bytes from
// unit AT on, unit n of all threads side by side.  (A run of units a thread
// would make every offset a constant, but copies whose 16-byte targets are
// scattered ran 1.35x slower.)
template <typename T, int V, int AT>
struct RingPieces {
  static constexpr int U = sizeof(T) / 2;
  static constexpr int END = AT + V * U;
  __device__ static __forceinline__ void fetch(uint4* stage, const T* row, const Place<true, 0>& p) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (p.in_row(v, 0)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          copy16(stage + (AT + v * U + u) * blockDim.x, reinterpret_cast<const uint4*>(row + p.column(v, 0)) + u);
      }
  }
  // zeros past the row's end
  __device__ static __forceinline__ Pairs read(const uint4* stage, int v, const Place<true, 0>& p) {
    Raw8<T> r{};
    if (p.in_row(v, 0)) {
#pragma unroll
      for (int u = 0; u < U; ++u) r.q[u] = stage[(AT + v * U + u) * blockDim.x];
    }
    return unpack(r);
  }
};

// Rows without 16-byte accesses: a row's threads copy the 16-byte granules that
// hold it, at the offset it has in them, and read it after a barrier.  (The
// first and last granule may hold bytes of the neighbouring rows or of what
// lies next to the array: memory is allocated in larger pieces, and nothing
// uses them.)
__host__ __device__ constexpr int linear_bytes(int H, int element) { return ((H * element + 30) >> 4) << 4; }
template <typename T>
__device__ __forceinline__ void copy_granules(char* region, const T* row, int H, int i, int lanes) {
  const int offset = (int)(reinterpret_cast<uintptr_t>(row) & 15);
  const char* from = reinterpret_cast<const char*>(row) - offset;
  const int units = (offset + H * (int)sizeof(T) + 15) >> 4;
  for (int u = i; u < units; u += lanes) copy16(region + 16 * u, from + 16 * u);
}
template <typename T>
__device__ __forceinline__ const T* in_granules(const char* region, const T* row) {
  return reinterpret_cast<const T*>(region + (reinterpret_cast<uintptr_t>(row) & 15));
}
template <bool WIDE>
__device__ __forceinline__ void row_barrier() {
  if constexpr (WIDE) __syncthreads();
  else __syncwarp();
}
// Rows in their ring: two if the widest rows of a kernel leave room for the
// CTAs that 512 threads make (elements: bytes of a column over all arrays).
__host__ __device__ constexpr int linear_stages(int columns, int lanes, int column_bytes, int arrays) {
  return 2 * (columns * column_bytes + 32 * arrays) * (512 / (lanes < 128 ? 128 : lanes)) *
                     (lanes < 128 ? 128 / lanes : 1) <= 224 * 1024
             ? 2
             : 1;
}

// Chunk v of a row in global memory, zeros past its end.
template <typename T, bool VEC, int LANES>
__device__ __forceinline__ Pairs load_pairs(const T* row, int v, const Place<VEC, LANES>& p) {
  if constexpr (VEC) {
    Raw8<T> r{};
    if (p.in_row(v, 0)) r = load_raw(row + p.column(v, 0));
    return unpack(r);
  } else {
    float x[8];
    if (p.in_row(v, 7)) {  // (all but a row's last warps)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = to_f32(row[p.column(v, k)]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = p.in_row(v, k) ? to_f32(row[p.column(v, k)]) : 0.0f;
    }
    Pairs o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.p[j] = make_float2(x[2 * j], x[2 * j + 1]);
    return o;
  }
}
template <typename T, bool VEC, int LANES>
__device__ __forceinline__ void put_pairs(T* row, int v, const Place<VEC, LANES>& p, const Pairs& x) {
  if constexpr (VEC) {
    if (p.in_row(v, 0)) store_pairs(row + p.column(v, 0), x);
  } else {
    if (p.in_row(v, 7)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) row[p.column(v, k)] = from_f32<T>(k & 1 ? x.p[k >> 1].y : x.p[k >> 1].x);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p.in_row(v, k)) row[p.column(v, k)] = from_f32<T>(k & 1 ? x.p[k >> 1].y : x.p[k >> 1].x);
    }
  }
}

// offset + w of chunk v, 1 without a weight; 0 past the row's end, where
// values taken off a mean are not zero.
template <typename T, bool VEC, int LANES>
__device__ __forceinline__ Pairs weight_pairs(const NormShape& s, const void* w, int v, const Place<VEC, LANES>& p) {
  Pairs o;
  float add = s.offset;
  if (!w) {
    add = 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.p[j] = both(0.0f);
  } else {
    o = s.weight_f32 ? load_pairs(static_cast<const float*>(w), v, p) : load_pairs(static_cast<const T*>(w), v, p);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o.p[j] = add2(o.p[j], make_float2(p.in_row(v, 2 * j) ? add : 0.0f, p.in_row(v, 2 * j + 1) ? add : 0.0f));
  return o;
}

// Adds a to the values within the row.
template <bool VEC, int LANES>
__device__ __forceinline__ void add_in_row(Pairs& x, float a, int v, const Place<VEC, LANES>& p) {
  if (p.in_row(v, 7)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x.p[j] = add2(x.p[j], both(a));
  } else if constexpr (!VEC) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p.in_row(v, 2 * j)) x.p[j].x += a;
      if (p.in_row(v, 2 * j + 1)) x.p[j].y += a;
    }
  }
}

__device__ __forceinline__ float gate_value(const NormShape& s, float g) {
  return s.gate_sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}
__device__ __forceinline__ void gate_pairs(const NormShape& s, Pairs& g) {
  if (s.gate_sigmoid) {
#pragma unroll
    for (int j = 0; j < 4; ++j) g.p[j] = make_float2(gate_value(s, g.p[j].x), gate_value(s, g.p[j].y));
  }
}

__device__ __forceinline__ float sum_pairs(float2 a) { return a.x + a.y; }

// A kernel's instantiation for a width: f(chunks, vec, constant lanes, wide).
// With 16-byte accesses a thread holds one chunk up to `narrow` columns, two
// up to 8192, four above; rows of up to 256 columns take a warp or less.
// Without, the row's threads are constants that leave few of them idle.
template <typename F>
cudaError_t with_width(int H, int narrow, bool vec, F&& f) {
  using std::integral_constant;
  constexpr auto one = integral_constant<int, 1>{};
  constexpr auto two = integral_constant<int, 2>{};
  constexpr auto four = integral_constant<int, 4>{};
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  if (vec) {
    constexpr auto any = integral_constant<int, 0>{};
    if (H <= 256) return f(one, yes, any, no);
    if (H <= narrow) return f(one, yes, any, yes);
    if (H <= 8192) return f(two, yes, any, yes);
    return f(four, yes, any, yes);
  }
  if (H <= 256) return f(one, no, integral_constant<int, 32>{}, no);
#define MOE_NORM_LANES(V, L) \
  if (H <= V::value * 8 * L) return f(V{}, no, integral_constant<int, L>{}, yes)
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  MOE_NORM_LANES(One, 64);
  MOE_NORM_LANES(One, 128);
  MOE_NORM_LANES(One, 192);
  MOE_NORM_LANES(One, 256);
  MOE_NORM_LANES(Two, 192);
  MOE_NORM_LANES(Two, 256);
  MOE_NORM_LANES(Two, 320);
  MOE_NORM_LANES(Two, 384);
  MOE_NORM_LANES(Two, 512);
#undef MOE_NORM_LANES
  return f(four, no, integral_constant<int, 512>{}, yes);
}

// Which parts a call has: a block output with both norms, only the pre-norm or
// only the post-norm (and, for the gradient, one of r'), or any.
constexpr int PARTS_ANY = 0, PARTS_ALL = 1, PARTS_PRE = 2, PARTS_POST = 3;
// with_gradient: of r' (true for the forward)
inline int parts_of(const NormShape& s, bool with_gradient) {
  if (!s.branch || !with_gradient) return PARTS_ANY;
  return s.post ? (s.pre ? PARTS_ALL : PARTS_POST) : s.pre ? PARTS_PRE : PARTS_ANY;
}
// Kinds of gate a kernel has code for, besides none and one value a token.
constexpr int GATE_BY_CHANNEL = 1, GATE_BY_ELEMENT = 2, GATE_ANY = 3;

// f(layer, gate, parts): the kernels for rows with 16-byte accesses come without
// the code of what a call leaves out, for both norms with any gate and for one
// norm with none or one value a token (8192 x 4096 bf16, only the pre-norm: the
// gradient 114 us with the code of all parts, 64 without); other calls
// share one that has it all, or all but a gate by channel or element.
template <bool VEC, int V, typename F>
cudaError_t with_kind(const NormShape& s, int parts, F&& f) {
  using std::integral_constant;
  if constexpr (VEC && V <= 2) {
    const bool by_element = s.gate == MOE_GATE_CHANNEL || s.gate == MOE_GATE_FULL;
    if (parts == PARTS_ALL && by_element) {
      auto gate = [&](auto layer) {
        constexpr auto all = integral_constant<int, PARTS_ALL>{};
        if (s.gate == MOE_GATE_CHANNEL) return f(layer, integral_constant<int, GATE_BY_CHANNEL>{}, all);
        return f(layer, integral_constant<int, GATE_BY_ELEMENT>{}, all);
      };
      return s.layer ? gate(std::true_type{}) : gate(std::false_type{});
    }
    if (parts != PARTS_ANY && !by_element) {
      auto kind = [&](auto some) {
        constexpr auto none = integral_constant<int, 0>{};
        return s.layer ? f(std::true_type{}, none, some) : f(std::false_type{}, none, some);
      };
      if (parts == PARTS_PRE) return kind(integral_constant<int, PARTS_PRE>{});
      if (parts == PARTS_POST) return kind(integral_constant<int, PARTS_POST>{});
      return kind(integral_constant<int, PARTS_ALL>{});
    }
  }
  constexpr auto any = integral_constant<int, PARTS_ANY>{};
  if constexpr (!VEC) {  // (whose registers the sums of a gate would overflow)
    if (s.gate == MOE_GATE_NONE || s.gate == MOE_GATE_TOKEN)
      return f(std::true_type{}, integral_constant<int, 0>{}, any);
  }
  return f(std::true_type{}, integral_constant<int, GATE_ANY>{}, any);
}

// Shared memory of an SM for the rings of n CTAs each: of 228 KB, less the
// runtime's 1 KB and the sums' words for each.
constexpr int SUMS_BYTES = RowSums<true>::WORDS * sizeof(float);
__host__ __device__ constexpr int ring_room(int n) { return (228 * 1024 / n - 1024 - SUMS_BYTES - 15) & ~15; }
constexpr int RING_ROOM = 226 * 1024;
static_assert(RING_ROOM + SUMS_BYTES <= 227 * 1024, "what a CTA may have");
// Rows in a ring: three keep two rows in flight.  Wide operands leave room for
// fewer, counted for 512 threads an SM.  (A constant: with a count known only
// at run time the forward ran 1.1x slower.)
__host__ __device__ constexpr int ring_stages(int units) {
  return units * 8192 * 3 <= RING_ROOM ? 3 : units * 8192 * 2 <= RING_ROOM ? 2 : 1;
}

// ---- the gradient's launch ----
// Sizes of the gradient's row loop, from the configuration alone (the
// workspace is sized by them without a device).
constexpr int BACKWARD_NARROW = 2048;
struct BackwardPlan {
  int lanes, threads, groups, ctas_per_sm, sums, hpad, smem;
  int64_t ctas(int64_t rows) const { return std::min<int64_t>((rows + groups - 1) / groups, 152 * ctas_per_sm); }
};

// units: of 16 bytes a thread has in a ring stage; linear_rows: stages of rows
// without 16-byte accesses.
inline BackwardPlan plan_backward(const moe_norm_config& c, bool vec, int V, int fixed_lanes, int units,
                                  int linear_rows) {
  BackwardPlan b{};
  b.lanes = row_lanes(c.hidden, V, fixed_lanes);
  b.threads = row_cta_threads(b.lanes);
  b.groups = rows_per_cta(b.lanes);
  b.sums = (c.branch && c.post) + (c.pre != 0) + (c.branch && c.gate == MOE_GATE_CHANNEL);
  b.hpad = (c.hidden + 7) & ~7;
  // (by the registers of the kernels' launch bounds)
  b.ctas_per_sm = 512 / b.threads;
  if (V == 4) {
    b.smem = b.sums * b.hpad * 4;  // the column sums
    return b;
  }
  // (the ring's memory serves to add the groups' column sums at the end)
  b.smem = b.groups > 1 ? b.sums * b.groups * b.hpad * 4 : 0;
  const int tb = c.dtype == MOE_DTYPE_F32 ? 4 : 2, rb = c.residual_dtype == MOE_DTYPE_F32 ? 4 : 2;
  const int arrays_t = (c.pre != 0) + (c.branch != 0) + (c.branch && c.gate == MOE_GATE_FULL);
  const int ring_bytes =
      vec ? ring_stages(units) * units * b.threads * 16
          : linear_rows * b.groups * (arrays_t * linear_bytes(c.hidden, tb) + 2 * linear_bytes(c.hidden, rb));
  while (b.ctas_per_sm > 1 && ring_bytes > ring_room(b.ctas_per_sm)) --b.ctas_per_sm;
  b.smem = std::max(b.smem, ring_bytes);
  return b;
}

// Units of 16 bytes a thread has in a stage of the gradient's ring: x and dr'
// of the residual's type, dh and y of the block's, and an element gate.
template <typename T, typename R, int V, bool WITH_GATE>
struct BackwardRun {
  using X = RingPieces<R, V, 0>;
  using D = RingPieces<R, V, X::END>;
  using DH = RingPieces<T, V, D::END>;
  using Y = RingPieces<T, V, DH::END>;
  using G = RingPieces<T, V, Y::END>;
  static constexpr int UNITS = WITH_GATE ? G::END : Y::END;
  __host__ __device__ static constexpr int linear(int lanes) {
    return lanes ? linear_stages(V * 8 * lanes, lanes, 3 * sizeof(T) + 2 * sizeof(R), 5) : 1;
  }
};

// The gradient's grid for a call: ctas of the kernel that serves it.
template <typename T, typename R>
int64_t gradient_ctas(const moe_norm_config& c, int64_t rows, bool vec, bool with_gradient) {
  const NormShape s = norm_shape(c);
  int64_t n = 0;
  with_width(c.hidden, BACKWARD_NARROW, vec, [&](auto chunks, auto v, auto fixed, auto) {
    constexpr int V = decltype(chunks)::value;
    constexpr bool VEC = decltype(v)::value;
    return with_kind<VEC, V>(s, parts_of(s, with_gradient), [&](auto, auto gate, auto) {
      using Run = BackwardRun<T, R, V, (decltype(gate)::value & GATE_BY_ELEMENT) != 0>;
      constexpr int LANES = decltype(fixed)::value;
      n = plan_backward(c, VEC, V, LANES, Run::UNITS, Run::linear(LANES)).ctas(rows);
      return cudaSuccess;
    });
  });
  return n;
}

// One translation unit each (norm_*.cu).
template <typename T, typename R>
cudaError_t launch_block_norm_t(const moe_norm_config& c, const moe_norm_io& io, int64_t rows, bool vec,
                                cudaStream_t stream);
template <typename T, typename R>
cudaError_t launch_block_norm_backward_t(const moe_norm_config& c, const moe_norm_grad_io& io, int64_t rows, bool vec,
                                         cudaStream_t stream);

}  // namespace moe
