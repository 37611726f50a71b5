// kernels_norm.cu - the norms before and after a block with its gate and
// residual, and their gradient.
//
//   u = n(y; wp), r' = r + a g u, h = n(r'; wn),
//   n(x; w) = (x - mean) rstd (offset + w), rstd = 1 / sqrt(mean((x - mean)^2) + eps),
// the mean taken as 0 for the RMS kind.  One CTA walks one row at a time;
// statistics come from the row's own values in a second pass (never as a
// difference of sums), in FP32.
#include "common.cuh"
#include "elem_types.cuh"
#include "kernels_ops.h"

namespace moe {

namespace {

struct NormShape {
  int H;
  bool layer, branch, post, pre, gate_sigmoid, weight_f32;
  int gate;
  float eps, offset, scale, inv_h;
};

// Sums over the CTA's threads of N values at a time: one barrier each, the
// partials double-buffered so that the next sum may start while slow threads
// still read this one.  Every thread gets the same bits.
struct RowSums {
  float* red;  // [2][4][32]
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= 4, "four sums at a time");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float* buf = red + (turn ^= 1) * 128;
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
      if (lane == 0) buf[n * 32 + warp] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = lane < warps ? buf[n * 32 + lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    }
  }
};

// Column of value k of this thread's chunk v: eight consecutive columns a
// thread where rows take 16-byte loads, else neighbouring threads on
// neighbouring columns.
template <bool VEC>
__device__ __forceinline__ int column(int v, int k) {
  return VEC ? (v * (int)blockDim.x + (int)threadIdx.x) * 8 + k
             : (v * 8 + k) * (int)blockDim.x + (int)threadIdx.x;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int v, int H, float (&o)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(v, 0);
    if (c < H) {
      load8(row + c, o);
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 0.0f;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column<false>(v, k);
      o[k] = c < H ? to_f32(row[c]) : 0.0f;
    }
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_chunk(T* row, int v, int H, const float (&x)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(v, 0);
    if (c < H) store8(row + c, x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column<false>(v, k);
      if (c < H) row[c] = from_f32<T>(x[k]);
    }
  }
}

// offset + w, or 1 without a weight.
template <bool VEC, typename T>
__device__ __forceinline__ void load_weight(const NormShape& s, const void* w, int v, float (&o)[8]) {
  if (!w) {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 1.0f;
    return;
  }
  if (s.weight_f32) load_chunk<VEC>(static_cast<const float*>(w), v, s.H, o);
  else load_chunk<VEC>(static_cast<const T*>(w), v, s.H, o);
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] += s.offset;
}

__device__ __forceinline__ float gate_value(const NormShape& s, float g) {
  return s.gate_sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// The gate's values for one chunk (1 without a gate).
template <bool VEC, typename T>
__device__ __forceinline__ void load_gate(const NormShape& s, const T* gate, int64_t stride, int64_t t, int v,
                                          float (&o)[8]) {
  if (s.gate == MOE_GATE_CHANNEL || s.gate == MOE_GATE_FULL) {
    load_chunk<VEC>(s.gate == MOE_GATE_FULL ? gate + t * stride : gate, v, s.H, o);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = gate_value(s, o[k]);
  } else {
    const float g = s.gate == MOE_GATE_TOKEN ? gate_value(s, to_f32(gate[t])) : 1.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = g;
  }
}

// Mean and 1 / sqrt(mean square + eps) of a row held in V chunks.
template <int V, bool VEC>
__device__ __forceinline__ void row_stats(const NormShape& s, RowSums& sums, const float (&x)[V][8], float& mean,
                                          float& rstd) {
  float a[1] = {0.0f};
  mean = 0.0f;
  if (s.layer) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) a[0] += column<VEC>(v, k) < s.H ? x[v][k] : 0.0f;
    sums(a);
    mean = a[0] * s.inv_h;
    a[0] = 0.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = x[v][k] - mean;
      if (column<VEC>(v, k) < s.H) a[0] = fmaf(d, d, a[0]);
    }
  sums(a);
  rstd = 1.0f / sqrtf(a[0] * s.inv_h + s.eps);
}

template <typename T, typename R, int V, bool VEC>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormShape s, const moe_norm_io io) {
  __shared__ float red[256];
  RowSums sums{red};
  const int64_t t = blockIdx.x;
  const R* rrow = static_cast<const R*>(io.residual) + t * io.residual_stride;
  float r[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) load_chunk<VEC>(rrow, v, s.H, r[v]);
  float mean, rstd;
  if (s.branch) {
    const T* yrow = static_cast<const T*>(io.y) + t * io.y_stride;
    float y[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) load_chunk<VEC>(yrow, v, s.H, y[v]);
    if (s.post) {
      row_stats<V, VEC>(s, sums, y, mean, rstd);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float w[8];
        load_weight<VEC, T>(s, io.post_weight, v, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[v][k] = (y[v][k] - mean) * rstd * w[k];
      }
    }
    R* out = static_cast<R*>(io.residual_out) + t * io.residual_out_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float g[8];
      load_gate<VEC>(s, static_cast<const T*>(io.gate), io.gate_stride, t, v, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[v][k] = fmaf(s.scale * g[k], y[v][k], r[v][k]);
      store_chunk<VEC>(out, v, s.H, r[v]);
    }
  }
  if (s.pre) {
    row_stats<V, VEC>(s, sums, r, mean, rstd);
    T* hrow = static_cast<T*>(io.h) + t * io.h_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w[8];
      load_weight<VEC, T>(s, io.pre_weight, v, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] *= (r[v][k] - mean) * rstd;
      store_chunk<VEC>(hrow, v, s.H, w);
    }
  }
}

// Column sums of the gradient, one FP32 row per kind in shared memory; a
// thread only ever touches its own columns, so no barrier is needed.
template <bool VEC>
__device__ __forceinline__ void add_columns(float* acc, int v, int H, const float (&x)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(v, 0);
    if (c >= H) return;
    float o[8];
    load8(acc + c, o);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] += x[k];
    store8(acc + c, o);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column<false>(v, k);
      if (c < H) acc[c] += x[k];
    }
  }
}

// Each CTA walks rows blockIdx.x, + gridDim.x, ...  With x = r' and
// a = dh (offset + wn):
//   dr = dr' + rstd_x (a - mean(a) - xhat mean(a xhat)),   dwn += dh xhat
// (mean(a) for LAYER only), and with e = branch_scale dr, b = e g (offset + wp):
//   dy = rstd_y (b - mean(b) - yhat mean(b yhat)),         dwp += e g yhat
//   dg = e u (summed over the row or the column as g is shared).
template <typename T, typename R, int V, bool VEC>
__global__ void __launch_bounds__(1024) block_norm_backward_kernel(const NormShape s, const moe_norm_grad_io io,
                                                                   int64_t rows, int n_sums, float* partial) {
  __shared__ float red[256];
  extern __shared__ __align__(16) float acc[];  // [n_sums][hpad]
  RowSums sums{red};
  const int H = s.H, hpad = (H + 7) & ~7;
  float* acc_post = acc;
  float* acc_pre = acc_post + (s.branch && s.post ? hpad : 0);
  float* acc_gate = acc_pre + (s.pre ? hpad : 0);
  for (int i = threadIdx.x; i < n_sums * hpad; i += blockDim.x) acc[i] = 0.0f;
  __syncthreads();

  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    const R* xrow = static_cast<const R*>(io.residual_out) + t * io.residual_out_stride;
    const T* dhrow = static_cast<const T*>(io.dh) + t * io.dh_stride;
    const R* drow = io.dresidual_out ? static_cast<const R*>(io.dresidual_out) + t * io.dresidual_out_stride : nullptr;
    const T* yrow = static_cast<const T*>(io.y) + t * io.y_stride;
    const T* gate = static_cast<const T*>(io.gate);
    const bool post = s.branch && s.post;
    float mx = 0.0f, my = 0.0f;
    if (s.layer && (s.pre || post)) {
      float a[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float x[8];
        if (s.pre) {
          load_chunk<VEC>(xrow, v, H, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[0] += x[k];
        }
        if (post) {
          load_chunk<VEC>(yrow, v, H, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[1] += x[k];
        }
      }
      sums(a);
      mx = a[0] * s.inv_h;
      my = a[1] * s.inv_h;
    }
    float rx = 0.0f, ry = 0.0f, ca = 0.0f, cx = 0.0f;
    if (s.pre || post) {
      float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // square sums of x and y; a; a (x - mean)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float x[8];
        if (s.pre) {
          float w[8], dh[8];
          load_chunk<VEC>(xrow, v, H, x);
          load_chunk<VEC>(dhrow, v, H, dh);
          load_weight<VEC, T>(s, io.pre_weight, v, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float d = x[k] - mx, a = dh[k] * w[k];
            if (column<VEC>(v, k) < H) {
              q[0] = fmaf(d, d, q[0]);
              q[2] += a;
              q[3] = fmaf(a, d, q[3]);
            }
          }
        }
        if (post) {
          load_chunk<VEC>(yrow, v, H, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float d = x[k] - my;
            if (column<VEC>(v, k) < H) q[1] = fmaf(d, d, q[1]);
          }
        }
      }
      sums(q);
      rx = 1.0f / sqrtf(q[0] * s.inv_h + s.eps);
      ry = 1.0f / sqrtf(q[1] * s.inv_h + s.eps);
      ca = s.layer ? q[2] * s.inv_h : 0.0f;
      cx = q[3] * rx * s.inv_h;  // mean(a xhat)
    }
    float dr[V][8];
    float q[3] = {0.0f, 0.0f, 0.0f};  // b; b yhat; e u (token gate)
    R* dres = static_cast<R*>(io.dresidual) + t * io.dresidual_stride;
    T* dyrow = static_cast<T*>(io.dy) + t * io.dy_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (drow) {
        load_chunk<VEC>(drow, v, H, dr[v]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) dr[v][k] = 0.0f;
      }
      if (s.pre) {
        float x[8], w[8], dh[8], dw[8];
        load_chunk<VEC>(xrow, v, H, x);
        load_chunk<VEC>(dhrow, v, H, dh);
        load_weight<VEC, T>(s, io.pre_weight, v, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xhat = (x[k] - mx) * rx;
          dr[v][k] += rx * (dh[k] * w[k] - ca - xhat * cx);
          dw[k] = dh[k] * xhat;
        }
        if (io.dpre_weight) add_columns<VEC>(acc_pre, v, H, dw);
      }
      store_chunk<VEC>(dres, v, H, dr[v]);
      if (!s.branch) continue;
      float y[8], w[8], g[8], dg[8];
      load_chunk<VEC>(yrow, v, H, y);
      load_gate<VEC>(s, gate, io.gate_stride, t, v, g);
      if (post) {
        load_weight<VEC, T>(s, io.post_weight, v, w);
        float dw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = s.scale * dr[v][k], yhat = (y[k] - my) * ry;
          const float eg = e * g[k];
          dw[k] = eg * yhat;
          if (column<VEC>(v, k) < H) {
            q[0] = fmaf(eg, w[k], q[0]);
            q[1] = fmaf(dw[k], w[k], q[1]);
            dg[k] = e * w[k] * yhat;
            q[2] += dg[k];
          }
        }
        if (io.dpost_weight) add_columns<VEC>(acc_post, v, H, dw);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = s.scale * dr[v][k];
          dg[k] = e * y[k];
          q[2] += dg[k];
          y[k] = e * g[k];
        }
        store_chunk<VEC>(dyrow, v, H, y);
      }
      if (io.dgate && (s.gate == MOE_GATE_CHANNEL || s.gate == MOE_GATE_FULL)) {
        if (s.gate_sigmoid) {
#pragma unroll
          for (int k = 0; k < 8; ++k) dg[k] *= g[k] * (1.0f - g[k]);
        }
        if (s.gate == MOE_GATE_CHANNEL) add_columns<VEC>(acc_gate, v, H, dg);
        else store_chunk<VEC>(static_cast<T*>(io.dgate) + t * io.dgate_stride, v, H, dg);
      }
    }
    if (!s.branch) continue;
    const bool token_gate = s.gate == MOE_GATE_TOKEN && io.dgate;
    if (post || token_gate) sums(q);
    if (token_gate && threadIdx.x == 0) {
      float d = q[2];
      if (s.gate_sigmoid) {
        const float g = gate_value(s, to_f32(gate[t]));
        d *= g * (1.0f - g);
      }
      static_cast<T*>(io.dgate)[t] = from_f32<T>(d);
    }
    if (!post) continue;
    const float cb = s.layer ? q[0] * s.inv_h : 0.0f, cy = q[1] * s.inv_h;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float y[8], w[8], g[8];
      load_chunk<VEC>(yrow, v, H, y);
      load_gate<VEC>(s, gate, io.gate_stride, t, v, g);
      load_weight<VEC, T>(s, io.post_weight, v, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float b = s.scale * dr[v][k] * g[k] * w[k];
        y[k] = ry * (b - cb - (y[k] - my) * ry * cy);
      }
      store_chunk<VEC>(dyrow, v, H, y);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_sums * hpad; i += blockDim.x)
    partial[(size_t)blockIdx.x * n_sums * hpad + i] = acc[i];
}

// Columns of the CTAs' partial sums, added in CTA order: 32 columns a CTA,
// 32 runs of rows, then a tree over the runs.
struct SumTargets {
  float* out[NORM_SUMS];
};
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int ctas, int n_sums,
                                                          int H, int hpad, SumTargets o) {
  __shared__ float tile[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
  float v = 0.0f;
  if (c < H)
    for (int b = threadIdx.y; b < ctas; b += 32) v += partial[((size_t)b * n_sums + which) * hpad + c];
  tile[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = tile[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  const int col = blockIdx.x * 32 + threadIdx.y;
  float* out = o.out[which];
  if (threadIdx.x == 0 && col < H && out) out[col] = v;
}

NormShape make_shape(const moe_norm_config& c) {
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

int row_threads(int H) {
  const int need = (H + 7) / 8;
  return need >= 1024 ? 1024 : (need + 31) / 32 * 32;
}

template <typename F>
cudaError_t with_types(const moe_norm_config& c, bool vec, F&& f) {
  using std::integral_constant;
  auto pick = [&](auto tv, auto rv) {
    const bool two = c.hidden > 8192;
    if (vec) return two ? f(tv, rv, integral_constant<int, 2>{}, std::true_type{})
                        : f(tv, rv, integral_constant<int, 1>{}, std::true_type{});
    return two ? f(tv, rv, integral_constant<int, 2>{}, std::false_type{})
               : f(tv, rv, integral_constant<int, 1>{}, std::false_type{});
  };
  const bool wide = c.residual_dtype == MOE_DTYPE_F32;
  if (c.dtype == MOE_DTYPE_F32) return pick(float(), float());
  if (c.dtype == MOE_DTYPE_F16) return wide ? pick(__half(), float()) : pick(__half(), __half());
  return wide ? pick(__nv_bfloat16(), float()) : pick(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace

cudaError_t launch_block_norm(const moe_norm_config& c, const moe_norm_io& io, int64_t rows, bool vec,
                              cudaStream_t s) {
  return with_types(c, vec, [&](auto tv, auto rv, auto v, auto vc) {
    return launch_k(block_norm_kernel<decltype(tv), decltype(rv), decltype(v)::value, decltype(vc)::value>,
                    dim3((unsigned)rows), dim3(row_threads(c.hidden)), 0, s, false, make_shape(c), io);
  });
}

int norm_backward_sums(const moe_norm_config& c) {
  return (c.branch && c.post) + (c.pre != 0) + (c.branch && c.gate == MOE_GATE_CHANNEL);
}

int norm_backward_ctas(const moe_norm_config& c, int64_t rows) {
  (void)c;
  return (int)(rows < 152 * 2 ? rows : 152 * 2);
}

cudaError_t launch_block_norm_backward(const moe_norm_config& c, const moe_norm_grad_io& io, int64_t rows, bool vec,
                                       cudaStream_t s) {
  const int ctas = norm_backward_ctas(c, rows), n_sums = norm_backward_sums(c);
  const int hpad = (c.hidden + 7) & ~7;
  const size_t smem = sizeof(float) * (size_t)n_sums * hpad;
  cudaError_t e = with_types(c, vec, [&](auto tv, auto rv, auto v, auto vc) {
    auto kernel = block_norm_backward_kernel<decltype(tv), decltype(rv), decltype(v)::value, decltype(vc)::value>;
    if (smem > 47 * 1024) {  // (1 KB of the default 48 KB is static)
      const cudaError_t a = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (a != cudaSuccess) return a;
    }
    return launch_k(kernel, dim3(ctas), dim3(row_threads(c.hidden)), smem, s, false, make_shape(c), io, rows, n_sums,
                    static_cast<float*>(io.workspace));
  });
  if (e != cudaSuccess || n_sums == 0) return e;
  SumTargets o{};
  int n = 0;
  if (c.branch && c.post) o.out[n++] = io.dpost_weight;
  if (c.pre) o.out[n++] = io.dpre_weight;
  if (c.branch && c.gate == MOE_GATE_CHANNEL) o.out[n++] = static_cast<float*>(io.dgate);
  return launch_k(column_sum_kernel, dim3((c.hidden + 31) / 32, n_sums), dim3(32, 32), 0, s, false,
                  static_cast<const float*>(io.workspace), ctas, n_sums, c.hidden, hpad, o);
}

}  // namespace moe
