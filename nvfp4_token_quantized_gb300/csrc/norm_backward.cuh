// norm_backward.cuh - the gradient of the norms around a block.
//
// With x = r', xc = x - mean (LAYER; else x) and a = dh (offset + wn):
//   dr = dr' + rstd_x (a - mean(a) - xc rstd_x^2 mean(a xc)),  dwn = sum over rows of dh xc rstd_x
// and with c = branch_scale, m = dr (offset + wp), yc as xc:
//   dy = c rstd_y (g m - mean(g m) - yc rstd_y^2 mean(g m yc)), dwp = sum over rows of c g dr yc rstd_y
//   dg = c m yc rstd_y, summed over the row or the column that shares g
// (the means of a and of g m for LAYER only; without a post-norm dy = c g dr
// and dg = c dr y).  A row takes three sums: the means, the squares with
// a xc, and g m yc.
//
// Bytes bound it: x, dh, dr', y come once (the passes over a row read it from
// the ring again), dr and dy leave once.  The column sums stay in the
// registers of the threads that own the columns while a CTA walks its rows;
// a second kernel adds the CTAs' sums in order.  16384 x 8192 bf16: 248 us, 6.5
// TB/s (column sums in shared memory and no ring: 730).  Centred rows with an
// element gate (4073 x 4096, FP32 residual): 86 us, 4.3 TB/s, bound by latency at
// the 16 warps an SM that their registers leave.  Rows above 8192 columns take
// four chunks a thread, whose sums lie in shared memory: 4096 x 12288 at 21 % of
// the copy rate.
#pragma once

#include "norm_common.cuh"

namespace moe {

namespace {

// Rows come through a ring, of pieces or of granules, up to two chunks a
// thread; wider ones from global memory, where L1 serves the later passes.
template <typename T, typename R, int V, bool VEC, int LANES, bool WIDE, bool LAYER, int GATE, int PARTS>
__global__ void __launch_bounds__(512, 1)
    block_norm_backward_kernel(const NormShape s, const moe_norm_grad_io io, int64_t rows, int n_sums,
                               int hpad, float* partial) {
  using Sums = RowSums<WIDE>;
  __shared__ __align__(16) float red[Sums::WORDS];
  extern __shared__ uint4 ring[];
  constexpr bool RING = VEC && V <= 2;
  constexpr bool LINEAR = !VEC && V <= 2;  // rows in granules
  constexpr bool KEEP = V <= 2;  // column sums and weights in registers
  using Run = BackwardRun<T, R, V, (GATE & GATE_BY_ELEMENT) != 0>;
  constexpr int STAGES = RING ? ring_stages(Run::UNITS) : 1;
  const int lanes = VEC ? s.lanes : LANES;
  Sums sums{red, lanes};
  sums.clear();
  const int groups = WIDE ? 1 : blockDim.x / lanes, group = WIDE ? 0 : threadIdx.x / lanes;
  const Place<VEC, LANES> p((int)threadIdx.x - group * lanes, lanes, s.H);
  const bool layer = LAYER && s.layer;
  const R* x_in = static_cast<const R*>(io.residual_out);
  const R* d_in = static_cast<const R*>(io.dresidual_out);
  const T* dh_in = static_cast<const T*>(io.dh);
  const T* y_in = static_cast<const T*>(io.y);
  const T* gate = static_cast<const T*>(io.gate);
  const bool branch = PARTS != PARTS_ANY || s.branch, has_d = PARTS != PARTS_ANY || d_in;
  const bool post = PARTS == PARTS_ANY ? s.post : PARTS != PARTS_PRE;
  const bool pre = PARTS == PARTS_ANY ? s.pre : PARTS != PARTS_POST;
  const bool full = (GATE & GATE_BY_ELEMENT) && (GATE != GATE_ANY || s.gate == MOE_GATE_FULL);
  const bool channel = (GATE & GATE_BY_CHANNEL) && (GATE != GATE_ANY || s.gate == MOE_GATE_CHANNEL);
  const bool by_element = full || channel, token = s.gate == MOE_GATE_TOKEN;
  // (without a post-norm y is needed for a gate's gradient only)
  const bool needs_y = branch && (post || (s.gate != MOE_GATE_NONE && io.dgate));

  Pairs sum_post[KEEP ? V : 1], sum_pre[KEEP ? V : 1], sum_gate[KEEP && (GATE & GATE_BY_CHANNEL) ? V : 1];
  Pairs wp[KEEP ? V : 1], wn[KEEP ? V : 1];
  float* acc = reinterpret_cast<float*>(ring);  // (not KEEP: [n_sums][hpad], each thread its own columns)
  float* acc_post = acc;
  float* acc_pre = acc_post + (post ? hpad : 0);
  float* acc_gate = acc_pre + (pre ? hpad : 0);
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum_post[v].p[j] = sum_pre[v].p[j] = both(0.0f);
        if constexpr (GATE & GATE_BY_CHANNEL) sum_gate[v].p[j] = both(0.0f);
      }
      if (post) wp[v] = weight_pairs<T>(s, io.post_weight, v, p);
      if (pre) wn[v] = weight_pairs<T>(s, io.pre_weight, v, p);
    }
  } else {
    for (int i = threadIdx.x; i < n_sums * hpad; i += blockDim.x) acc[i] = 0.0f;
    __syncthreads();
  }
  auto post_w = [&](int v) {
    if constexpr (KEEP) return wp[v];
    else return weight_pairs<T>(s, io.post_weight, v, p);
  };
  auto pre_w = [&](int v) {
    if constexpr (KEEP) return wn[v];
    else return weight_pairs<T>(s, io.pre_weight, v, p);
  };
  // adds f x to this thread's columns of one sum
  auto add_columns = [&](Pairs& mine, float* row, int v, const Pairs& x, float f) {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < 4; ++j) mine.p[j] = fma2(x.p[j], both(f), mine.p[j]);
    } else {
      Pairs o = load_pairs<float>(row, v, p);
#pragma unroll
      for (int j = 0; j < 4; ++j) o.p[j] = fma2(x.p[j], both(f), o.p[j]);
      put_pairs<float>(row, v, p, o);
    }
  };
  // takes a mean off the values within the row
  auto centre = [&](Pairs& x, int v, float mean) {
    if (layer) add_in_row(x, -mean, v, p);
  };

  const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups;
  const int warp_group = WIDE ? 0 : (threadIdx.x & ~31) / lanes;
  auto run_of = [&](int stage) { return ring + stage * Run::UNITS * blockDim.x + threadIdx.x; };
  constexpr int ROWS = Run::linear(LANES);
  const int r_bytes = linear_bytes(s.H, sizeof(R)), t_bytes = linear_bytes(s.H, sizeof(T));
  const int linear_row = 2 * r_bytes + ((pre ? 1 : 0) + (branch ? 1 : 0) + (full ? 1 : 0)) * t_bytes;
  const int at_dh = 2 * r_bytes, at_y = at_dh + (pre ? t_bytes : 0), at_gate = at_y + (branch ? t_bytes : 0);
  auto region_of = [&](int stage) { return reinterpret_cast<char*>(ring) + (stage * groups + group) * linear_row; };
  auto fetch = [&](int64_t t, int stage) {
    if constexpr (LINEAR) {
      if (t < rows) {
        char* region = region_of(stage);
        if (pre) {
          copy_granules(region, x_in + t * io.residual_out_stride, s.H, p.i, LANES);
          copy_granules(region + at_dh, dh_in + t * io.dh_stride, s.H, p.i, LANES);
        }
        if (has_d) copy_granules(region + r_bytes, d_in + t * io.dresidual_out_stride, s.H, p.i, LANES);
        if (needs_y) copy_granules(region + at_y, y_in + t * io.y_stride, s.H, p.i, LANES);
        if (full) copy_granules(region + at_gate, gate + t * io.gate_stride, s.H, p.i, LANES);
      }
      copies_commit();
    }
    if constexpr (RING) {
      if (t < rows) {
        uint4* run = run_of(stage);
        if (pre) {
          Run::X::fetch(run, x_in + t * io.residual_out_stride, p);
          Run::DH::fetch(run, dh_in + t * io.dh_stride, p);
        }
        if (has_d) Run::D::fetch(run, d_in + t * io.dresidual_out_stride, p);
        if (needs_y) Run::Y::fetch(run, y_in + t * io.y_stride, p);
        if (full) Run::G::fetch(run, gate + t * io.gate_stride, p);
      }
      copies_commit();
    }
  };
  int64_t t = first + group;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(t + i * step, i);
  if constexpr (LINEAR && ROWS == 2) fetch(t, 0);
  int stage = 0;
#pragma unroll 1
  for (int64_t w = first + warp_group; w < rows; w += step, t += step) {
    const bool live = WIDE || t < rows;
    const uint4* run = run_of(stage);
    if constexpr (RING) {
      fetch(t + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
      copies_wait<STAGES - 1>();
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // the rows (the last one where this group has none)
    const int64_t tr = live ? t : rows - 1;
    const R* x_row = x_in + tr * io.residual_out_stride;
    const R* d_row = d_in + tr * io.dresidual_out_stride;
    const T* dh_row = dh_in + tr * io.dh_stride;
    const T* y_row = y_in + tr * io.y_stride;
    const T* g_row = gate + tr * io.gate_stride;
    if constexpr (LINEAR) {
      const char* region = region_of(stage);
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
      x_row = in_granules(region, x_row);
      d_row = in_granules(region + r_bytes, d_row);
      dh_row = in_granules(region + at_dh, dh_row);
      y_row = in_granules(region + at_y, y_row);
      g_row = in_granules(region + at_gate, g_row);
    }
    auto get_x = [&](int v) {
      if constexpr (RING) return Run::X::read(run, v, p);
      else return load_pairs<R>(x_row, v, p);
    };
    auto get_d = [&](int v) {
      if constexpr (RING) return Run::D::read(run, v, p);
      else return load_pairs<R>(d_row, v, p);
    };
    auto get_dh = [&](int v) {
      if constexpr (RING) return Run::DH::read(run, v, p);
      else return load_pairs<T>(dh_row, v, p);
    };
    auto get_y = [&](int v) {
      if constexpr (RING) return Run::Y::read(run, v, p);
      else return load_pairs<T>(y_row, v, p);
    };
    auto get_gate = [&](int v) {
      Pairs g;
      if (!full) g = load_pairs<T>(gate, v, p);
      else if constexpr (RING) g = Run::G::read(run, v, p);
      else g = load_pairs<T>(g_row, v, p);
      gate_pairs(s, g);
      return g;
    };
    float mx = 0.0f, my = 0.0f;
    if (layer) {
      if (pre || post) {
        float2 a = both(0.0f), b = both(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (pre) {
            const Pairs x = get_x(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) a = add2(a, x.p[j]);
          }
          if (post) {
            const Pairs y = get_y(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) b = add2(b, y.p[j]);
          }
        }
        float q[2] = {sum_pairs(a), sum_pairs(b)};
        sums(q);
        mx = q[0] * s.inv_h;
        my = q[1] * s.inv_h;
      }
    }
    float rx = 0.0f, ry = 0.0f, mean_a = 0.0f, along_x = 0.0f;
    if (pre || post) {
      float2 xx = both(0.0f), yy = both(0.0f), sa = both(0.0f), ax = both(0.0f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (pre) {
          Pairs x = get_x(v);
          const Pairs dh = get_dh(v), f = pre_w(v);
          centre(x, v, mx);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = mul2(dh.p[j], f.p[j]);
            xx = fma2(x.p[j], x.p[j], xx);
            ax = fma2(a, x.p[j], ax);
            if (LAYER) sa = add2(sa, a);
          }
        }
        if (post) {
          Pairs y = get_y(v);
          centre(y, v, my);
#pragma unroll
          for (int j = 0; j < 4; ++j) yy = fma2(y.p[j], y.p[j], yy);
        }
      }
      if constexpr (PARTS == PARTS_POST) {
        float q[1] = {sum_pairs(yy)};
        sums(q);
        yy.x = q[0];
      } else if constexpr (PARTS == PARTS_PRE && !LAYER) {
        float q[2] = {sum_pairs(xx), sum_pairs(ax)};
        sums(q);
        xx.x = q[0], ax.x = q[1];
      } else if constexpr (LAYER) {
        float q[4] = {sum_pairs(xx), sum_pairs(yy), sum_pairs(ax), sum_pairs(sa)};
        sums(q);
        xx.x = q[0], yy.x = q[1], ax.x = q[2];
        if (layer) mean_a = q[3] * s.inv_h;
      } else {
        float q[4] = {sum_pairs(xx), sum_pairs(yy), sum_pairs(ax), 0.0f};
        sums(q);
        xx.x = q[0], yy.x = q[1], ax.x = q[2];
      }
      rx = inv_sqrt(xx.x * s.inv_h + s.eps);
      ry = inv_sqrt(yy.x * s.inv_h + s.eps);
      along_x = ax.x * s.inv_h * rx * rx * rx;
    }
    float c = s.scale, g_token = 1.0f;
    if (token) {
      g_token = gate_value(s, to_f32(gate[tr]));
      c *= g_token;
    }
    Pairs dr[V];
    float2 gm = both(0.0f), gmy = both(0.0f);  // sums of g m and g m yc (a token's gate left out)
    R* dres = static_cast<R*>(io.dresidual) + t * io.dresidual_stride;
    T* dyrow = static_cast<T*>(io.dy) + t * io.dy_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (has_d) {
        dr[v] = get_d(v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) dr[v].p[j] = both(0.0f);
      }
      if (pre) {
        Pairs x = get_x(v);
        Pairs dh = get_dh(v);
        const Pairs f = pre_w(v);
        centre(x, v, mx);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 a = mul2(dh.p[j], f.p[j]);
          if constexpr (LAYER) a = add2(a, both(-mean_a));
          dr[v].p[j] = fma2(a, both(rx), dr[v].p[j]);
          dr[v].p[j] = fma2(x.p[j], both(-along_x), dr[v].p[j]);
          dh.p[j] = mul2(dh.p[j], x.p[j]);
        }
        if (live) add_columns(sum_pre[KEEP ? v : 0], acc_pre, v, dh, rx);
      }
      if (live) put_pairs<R>(dres, v, p, dr[v]);
      if (!branch) continue;
      Pairs y;
      if (needs_y) {
        y = get_y(v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y.p[j] = both(0.0f);
      }
      if (!post) {
        Pairs g;
        if (by_element) g = get_gate(v);
        Pairs dy;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dy.p[j] = mul2(dr[v].p[j], both(c));
          y.p[j] = mul2(dr[v].p[j], y.p[j]);
          gmy = add2(gmy, y.p[j]);
          if (by_element) dy.p[j] = mul2(dy.p[j], g.p[j]);
        }
        if (live) put_pairs<T>(dyrow, v, p, dy);
        if (by_element && io.dgate) {
          if (s.gate_sigmoid) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y.p[j] = mul2(y.p[j], make_float2(g.p[j].x * (1.0f - g.p[j].x), g.p[j].y * (1.0f - g.p[j].y)));
          }
          if (channel) {
            if (live) add_columns(sum_gate[KEEP && (GATE & GATE_BY_CHANNEL) ? v : 0], acc_gate, v, y, s.scale);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) y.p[j] = mul2(y.p[j], both(s.scale));
            if (live) put_pairs<T>(static_cast<T*>(io.dgate) + t * io.dgate_stride, v, p, y);
          }
        }
        continue;
      }
      const Pairs f = post_w(v);
      centre(y, v, my);
      Pairs g;
      if (by_element) g = get_gate(v);
      Pairs dy;  // dr yc, then m yc
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dy.p[j] = mul2(dr[v].p[j], y.p[j]);
        float2 m = mul2(dr[v].p[j], f.p[j]), my2 = mul2(dy.p[j], f.p[j]);
        if (by_element) {
          dy.p[j] = mul2(dy.p[j], g.p[j]);  // (g dr yc: the weight's)
          y.p[j] = my2;
          m = mul2(m, g.p[j]);
          my2 = mul2(my2, g.p[j]);
        }
        if constexpr (LAYER) gm = add2(gm, m);
        gmy = add2(gmy, my2);
      }
      if (live) add_columns(sum_post[KEEP ? v : 0], acc_post, v, dy, c * ry);
      if (by_element && io.dgate) {
        if (s.gate_sigmoid) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y.p[j] = mul2(y.p[j], make_float2(g.p[j].x * (1.0f - g.p[j].x), g.p[j].y * (1.0f - g.p[j].y)));
        }
        if (channel) {
          if (live) add_columns(sum_gate[KEEP && (GATE & GATE_BY_CHANNEL) ? v : 0], acc_gate, v, y, s.scale * ry);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) y.p[j] = mul2(y.p[j], both(s.scale * ry));
          if (live) put_pairs<T>(static_cast<T*>(io.dgate) + t * io.dgate_stride, v, p, y);
        }
      }
    }
    if (!post && !token) continue;
    float q[2] = {sum_pairs(gmy), LAYER ? sum_pairs(gm) : 0.0f};
    if constexpr (LAYER) {
      sums(q);
    } else {
      float q1[1] = {q[0]};
      sums(q1);
      q[0] = q1[0];
    }
    if (token && io.dgate && live && p.i == 0) {
      float d = s.scale * (post ? ry : 1.0f) * q[0];
      if (s.gate_sigmoid) d *= g_token * (1.0f - g_token);
      static_cast<T*>(io.dgate)[t] = from_f32<T>(d);
    }
    if (!post) continue;
    const float k = c * ry, mean_gm = layer ? q[1] * s.inv_h * k : 0.0f, along_y = q[0] * s.inv_h * k * ry * ry;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Pairs y = get_y(v);
      const Pairs f = post_w(v);
      centre(y, v, my);
      Pairs g;
      if (by_element) g = get_gate(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 m = mul2(dr[v].p[j], f.p[j]);
        if (by_element) m = mul2(m, g.p[j]);
        float2 d = mul2(y.p[j], both(-along_y));
        if constexpr (LAYER) d = add2(d, both(-mean_gm));
        y.p[j] = fma2(m, both(k), d);
      }
      if (live) put_pairs<T>(dyrow, v, p, y);
    }
  }
  copies_wait<0>();
  pdl_trigger();
  if (n_sums == 0) return;
  float* out = partial + (size_t)blockIdx.x * n_sums * hpad;
  if constexpr (!KEEP) {
    __syncthreads();
    for (int i = threadIdx.x; i < n_sums * hpad; i += blockDim.x) out[i] = acc[i];
  } else {
    // straight to the CTA's row of partial sums, or, where the CTA has
    // several groups, into shared memory and added in group order
    float* to = out;
    if (groups > 1) {
      __syncthreads();  // (the ring is idle)
      to = acc + (size_t)group * n_sums * hpad;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float* row = to;
      if (post) {
        put_pairs<float>(row, v, p, sum_post[v]);
        row += hpad;
      }
      if (pre) {
        put_pairs<float>(row, v, p, sum_pre[v]);
        row += hpad;
      }
      if (channel) put_pairs<float>(row, v, p, sum_gate[KEEP && (GATE & GATE_BY_CHANNEL) ? v : 0]);
    }
    if (groups > 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n_sums * hpad; i += blockDim.x) {
        float a = 0.0f;
        for (int g = 0; g < groups; ++g) a += acc[(size_t)g * n_sums * hpad + i];
        out[i] = a;
      }
    }
  }
}

template <typename T, typename R, int V, bool VEC, int LANES, bool WIDE, bool LAYER, int GATE, int PARTS>
cudaError_t launch_gradient_rows(const moe_norm_config& c, NormShape s, const moe_norm_grad_io& io, int64_t rows,
                                 cudaStream_t stream) {
  using Run = BackwardRun<T, R, V, (GATE & GATE_BY_ELEMENT) != 0>;
  const BackwardPlan b = plan_backward(c, VEC, V, LANES, Run::UNITS, Run::linear(LANES));
  s.lanes = b.lanes;
  auto kernel = block_norm_backward_kernel<T, R, V, VEC, LANES, WIDE, LAYER, GATE, PARTS>;
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e = raise_shared(kernel, RING_ROOM, raised);
  if (e != cudaSuccess) return e;
  return launch_k(kernel, dim3((unsigned)b.ctas(rows)), dim3(b.threads), b.smem, stream, false, s, io, rows, b.sums,
                  b.hpad, static_cast<float*>(io.workspace));
}

}  // namespace

template <typename T, typename R>
cudaError_t launch_block_norm_backward_t(const moe_norm_config& c, const moe_norm_grad_io& io, int64_t rows, bool vec,
                                         cudaStream_t stream) {
  const NormShape s = norm_shape(c);
  return with_width(s.H, BACKWARD_NARROW, vec, [&](auto chunks, auto v, auto fixed, auto wide) {
    constexpr int V = decltype(chunks)::value;
    constexpr bool VEC = decltype(v)::value;
    return with_kind<VEC, V>(s, parts_of(s, io.dresidual_out != nullptr), [&](auto layer, auto gate, auto parts) {
      return launch_gradient_rows<T, R, V, VEC, decltype(fixed)::value, decltype(wide)::value, decltype(layer)::value,
                                  decltype(gate)::value, decltype(parts)::value>(c, s, io, rows, stream);
    });
  });
}

}  // namespace moe
