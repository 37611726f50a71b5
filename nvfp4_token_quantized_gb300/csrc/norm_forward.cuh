// norm_forward.cuh - the norms before and after a block with its gate and
// residual.
//
//   u = n(y; wp), r' = r + a g u, h = n(r'; wn),
//   n(x; w) = (x - mean) rstd (offset + w), rstd = 1 / sqrt(mean((x - mean)^2) + eps),
// the mean taken as 0 for the RMS kind.  Statistics come from the row's own
// values after the mean has been taken off (never as a difference of sums),
// in FP32.
//
// Bytes bound it: y, r, r' and h move once, a row stays on the SM between its
// two sums.  Rows arrive two ahead of the arithmetic by asynchronous copies, each
// thread its own pieces (no barrier), and their sums take one barrier each.
// 16384 x 8192 bf16: 165 us, 6.5 TB/s (one row a CTA of 1024 threads: 407); 4096
// x 2048 with an FP32 residual and a gate by channel: 21 us, 4.8 TB/s; a single
// row of 2048: 2.4 us, a launch and two sums.
#pragma once

#include "norm_common.cuh"

namespace moe {

namespace {

// Takes the mean of a row off (LAYER) and returns 1 / sqrt(mean square + eps).
template <int V, bool LAYER, bool VEC, int LANES, typename Sums>
__device__ __forceinline__ float centre_and_scale(const NormShape& s, const Place<VEC, LANES>& p, Sums& sums,
                                                  Pairs (&x)[V]) {
  float a[1];
  if (LAYER && s.layer) {
    float2 t = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) t = add2(t, x[v].p[j]);
    a[0] = sum_pairs(t);
    sums(a);
    const float mean = -a[0] * s.inv_h;
#pragma unroll
    for (int v = 0; v < V; ++v) add_in_row(x[v], mean, v, p);
  }
  float2 q = both(0.0f);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) q = fma2(x[v].p[j], x[v].p[j], q);
  a[0] = sum_pairs(q);
  sums(a);
  return inv_sqrt(a[0] * s.inv_h + s.eps);
}

template <typename T, typename R, int V, bool WITH_GATE>
struct ForwardRun {
  using X = RingPieces<R, V, 0>;
  using Y = RingPieces<T, V, X::END>;
  using G = RingPieces<T, V, Y::END>;
  static constexpr int UNITS = WITH_GATE ? G::END : Y::END;
  __host__ __device__ static constexpr int linear(int lanes) {
    return lanes ? linear_stages(V * 8 * lanes, lanes, 2 * sizeof(T) + sizeof(R), 3) : 1;
  }
};

// A group of s.lanes threads walks rows; each CTA holds blockDim.x / s.lanes
// groups.  LAYER, GATE and PARTS leave the code of the centred kind, of gates
// and of absent parts out.
template <typename T, typename R, int V, bool VEC, int LANES, bool WIDE, bool LAYER, int GATE, int PARTS>
__global__ void __launch_bounds__(512, V == 1 ? 2 : 1) block_norm_kernel(const NormShape s, const moe_norm_io io,
                                                                         int64_t rows) {
  using Run = ForwardRun<T, R, V, (GATE & GATE_BY_ELEMENT) != 0>;
  constexpr int STAGES = ring_stages(Run::UNITS);
  using Sums = RowSums<WIDE>;
  __shared__ __align__(16) float red[Sums::WORDS];
  extern __shared__ uint4 ring[];
  const int lanes = VEC ? s.lanes : LANES;
  Sums sums{red, lanes};
  sums.clear();
  const int groups = WIDE ? 1 : blockDim.x / lanes, group = WIDE ? 0 : threadIdx.x / lanes;
  const Place<VEC, LANES> p((int)threadIdx.x - group * lanes, lanes, s.H);
  const bool branch = PARTS != PARTS_ANY || s.branch;
  const bool post = PARTS == PARTS_ANY ? s.post : PARTS != PARTS_PRE;
  const bool pre = PARTS == PARTS_ANY ? s.pre : PARTS != PARTS_POST;
  const bool full = (GATE & GATE_BY_ELEMENT) && (GATE != GATE_ANY || s.gate == MOE_GATE_FULL);
  const bool channel = (GATE & GATE_BY_CHANNEL) && (GATE != GATE_ANY || s.gate == MOE_GATE_CHANNEL);
  const bool by_element = full || channel, token = s.gate == MOE_GATE_TOKEN;
  const T* gate = static_cast<const T*>(io.gate);
  // The weights stay in registers while two chunks' worth fit there; wider
  // rows read them again for each row (L1 and L2 hold them).
  constexpr bool KEEP = V <= 2;
  Pairs wp[KEEP ? V : 1], wn[KEEP ? V : 1];
  const int64_t step = (int64_t)gridDim.x * groups;
  // (the rows of a warp end together: a group past the last row idles)
  const int64_t first = (int64_t)blockIdx.x * groups;
  const int warp_group = WIDE ? 0 : (threadIdx.x & ~31) / lanes;

  // Rows without 16-byte accesses lie in granules; the widest stay in global
  // memory.
  constexpr bool LINEAR = !VEC && V <= 2;
  constexpr int ROWS = Run::linear(LANES);
  const int r_bytes = linear_bytes(s.H, sizeof(R)), t_bytes = linear_bytes(s.H, sizeof(T));
  const int linear_row = r_bytes + ((branch ? 1 : 0) + (full ? 1 : 0)) * t_bytes;
  auto run_of = [&](int stage) { return ring + stage * Run::UNITS * blockDim.x + threadIdx.x; };
  auto region_of = [&](int stage) { return reinterpret_cast<char*>(ring) + (stage * groups + group) * linear_row; };
  auto r_row = [&](int64_t t) { return static_cast<const R*>(io.residual) + t * io.residual_stride; };
  auto y_row = [&](int64_t t) { return static_cast<const T*>(io.y) + t * io.y_stride; };
  auto g_row = [&](int64_t t) { return gate + t * io.gate_stride; };
  auto fetch = [&](int64_t t, int stage) {
    if constexpr (VEC) {
      if (t < rows) {
        uint4* run = run_of(stage);
        Run::X::fetch(run, r_row(t), p);
        if (branch) Run::Y::fetch(run, y_row(t), p);
        if (full) Run::G::fetch(run, g_row(t), p);
      }
      copies_commit();
    } else if constexpr (LINEAR) {
      if (t < rows) {
        char* region = region_of(stage);
        copy_granules(region, r_row(t), s.H, p.i, LANES);
        if (branch) copy_granules(region + r_bytes, y_row(t), s.H, p.i, LANES);
        if (full) copy_granules(region + r_bytes + t_bytes, g_row(t), s.H, p.i, LANES);
      }
      copies_commit();
    }
  };
  int64_t t = first + group;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(t + i * step, i);
  } else if constexpr (LINEAR && ROWS == 2) {
    fetch(t, 0);
  }
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (post) wp[v] = weight_pairs<T>(s, io.post_weight, v, p);
      if (pre) wn[v] = weight_pairs<T>(s, io.pre_weight, v, p);
    }
  }
  int stage = 0;
#pragma unroll 1
  for (int64_t w = first + warp_group; w < rows; w += step, t += step) {
    const bool live = WIDE || t < rows;
    const uint4* run = run_of(stage);
    Pairs r[V], y[V];
    const T* from_gate = nullptr;
    if constexpr (VEC) {
      // into the stage of the row before this one (or, with one stage, this
      // row's), whose values this thread has used
      fetch(t + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
      copies_wait<STAGES - 1>();
      stage = stage + 1 == STAGES ? 0 : stage + 1;
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] = Run::X::read(run, v, p);
      if (branch) {
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = Run::Y::read(run, v, p);
      }
    } else {
      const int64_t tr = live ? t : rows - 1;
      const R* from_r = r_row(tr);
      const T* from_y = y_row(tr);
      from_gate = g_row(tr);
      if constexpr (LINEAR) {
        char* region = region_of(stage);
        if constexpr (ROWS == 2) {
          // this row has landed for all its threads, who have left the other stage
          copies_wait<0>();
          row_barrier<WIDE>();
          fetch(t + step, stage ^ 1);
          stage ^= 1;
        } else {
          row_barrier<WIDE>();
          fetch(t, 0);
          copies_wait<0>();
          row_barrier<WIDE>();
        }
        from_r = in_granules(region, from_r);
        from_y = in_granules(region + r_bytes, from_y);
        from_gate = in_granules(region + r_bytes + t_bytes, from_gate);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        r[v] = load_pairs<R>(from_r, v, p);
        if (branch) y[v] = load_pairs<T>(from_y, v, p);
      }
    }
    if (branch) {
      float scale = s.scale;
      if (token && live) scale *= gate_value(s, to_f32(gate[t]));
      if (post) scale *= centre_and_scale<V, LAYER>(s, p, sums, y);
      const float2 k = both(scale);
      R* out = static_cast<R*>(io.residual_out) + t * io.residual_out_stride;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (post) {
          const Pairs f = KEEP ? wp[KEEP ? v : 0] : weight_pairs<T>(s, io.post_weight, v, p);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[v].p[j] = mul2(y[v].p[j], f.p[j]);
        }
        if (by_element && live) {
          Pairs g;
          if (!full) g = load_pairs<T>(gate, v, p);
          else if constexpr (VEC) g = Run::G::read(run, v, p);
          else g = load_pairs<T>(from_gate, v, p);
          gate_pairs(s, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[v].p[j] = mul2(y[v].p[j], g.p[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r[v].p[j] = fma2(y[v].p[j], k, r[v].p[j]);
        if (live) put_pairs<R>(out, v, p, r[v]);
      }
    }
    if (pre) {
      const float2 k = both(centre_and_scale<V, LAYER>(s, p, sums, r));
      T* h = static_cast<T*>(io.h) + t * io.h_stride;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Pairs f = KEEP ? wn[KEEP ? v : 0] : weight_pairs<T>(s, io.pre_weight, v, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(mul2(r[v].p[j], k), f.p[j]);
        if (live) put_pairs<T>(h, v, p, r[v]);
      }
    }
  }
  copies_wait<0>();
}

template <typename T, typename R, int V, bool VEC, int LANES, bool WIDE, bool LAYER, int GATE, int PARTS>
cudaError_t launch_rows(NormShape s, const moe_norm_io& io, int64_t rows, cudaStream_t stream) {
  s.lanes = row_lanes(s.H, V, LANES);
  const int threads = row_cta_threads(s.lanes), groups = rows_per_cta(s.lanes);
  using Run = ForwardRun<T, R, V, (GATE & GATE_BY_ELEMENT) != 0>;
  constexpr int UNITS = Run::UNITS;
  constexpr bool LINEAR = !VEC && V <= 2;
  const int linear_row = linear_bytes(s.H, sizeof(R)) +
                         (s.branch + (s.gate == MOE_GATE_FULL)) * linear_bytes(s.H, sizeof(T));
  const int smem = VEC      ? ring_stages(UNITS) * UNITS * threads * 16
                   : LINEAR ? Run::linear(LANES) * groups * linear_row
                            : 0;
  auto kernel = block_norm_kernel<T, R, V, VEC, LANES, WIDE, LAYER, GATE, PARTS>;
  static std::atomic<uint64_t> raised{0};
  static std::atomic<int> resident[17];  // CTAs an SM holds, by warps; 0: not asked yet
  cudaError_t e = raise_shared(kernel, VEC || LINEAR ? RING_ROOM : 0, raised);
  if (e != cudaSuccess) return e;
  std::atomic<int>& slot = resident[threads / 32];
  int ctas = slot.load(std::memory_order_relaxed);
  if (ctas == 0) {
    // (granules: of the widest rows the kernel serves)
    constexpr int WIDEST = V * 8 * LANES;
    const int most = LINEAR ? Run::linear(LANES) * groups *
                                  (linear_bytes(WIDEST, sizeof(R)) + 2 * linear_bytes(WIDEST, sizeof(T)))
                            : smem;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, threads, most);
    if (e != cudaSuccess) return e;
    ctas = std::max(ctas, 1);
    slot.store(ctas, std::memory_order_relaxed);
  }
  const int64_t need = (rows + groups - 1) / groups;
  return launch_k(kernel, dim3((unsigned)std::min<int64_t>(need, 152 * ctas)), dim3(threads), smem, stream, false, s,
                  io, rows);
}

}  // namespace

template <typename T, typename R>
cudaError_t launch_block_norm_t(const moe_norm_config& c, const moe_norm_io& io, int64_t rows, bool vec,
                                cudaStream_t stream) {
  const NormShape s = norm_shape(c);
  return with_width(s.H, 4096, vec, [&](auto chunks, auto v, auto fixed, auto wide) {
    constexpr int V = decltype(chunks)::value;
    constexpr bool VEC = decltype(v)::value;
    return with_kind<VEC, V>(s, parts_of(s, true), [&](auto layer, auto gate, auto parts) {
      return launch_rows<T, R, V, VEC, decltype(fixed)::value, decltype(wide)::value, decltype(layer)::value,
                         decltype(gate)::value, decltype(parts)::value>(s, io, rows, stream);
    });
  });
}

}  // namespace moe
