// kernels_norm.cu - the block norms' launches by element type, and the second
// kernel of their gradient.
#include "norm_common.cuh"

namespace moe {

namespace {

// Columns of the CTAs' partial sums, added in an order fixed by their
// number: 32 columns a CTA, 32 runs of rows, then a tree over the runs.
struct SumTargets {
  float* out[NORM_SUMS];
};
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int ctas, int n_sums,
                                                          int H, int hpad, SumTargets o) {
  __shared__ float tile[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
  pdl_wait();
  float v = 0.0f;
  if (c < H)
    for (int b = threadIdx.y; b < ctas; b += 32) v += __ldcg(partial + ((size_t)b * n_sums + which) * hpad + c);
  tile[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = tile[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  const int col = blockIdx.x * 32 + threadIdx.y;
  float* out = o.out[which];
  if (threadIdx.x == 0 && col < H && out) out[col] = v;
}

// f(T, R): the element types of a configuration.
template <typename F>
cudaError_t with_types(const moe_norm_config& c, F&& f) {
  const bool wide = c.residual_dtype == MOE_DTYPE_F32;
  if (c.dtype == MOE_DTYPE_F32) return f(float(), float());
  if (c.dtype == MOE_DTYPE_F16) return wide ? f(__half(), float()) : f(__half(), __half());
  return wide ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
}

int64_t plan_ctas(const moe_norm_config& c, int64_t rows, bool vec, bool with_gradient) {
  int64_t n = 0;
  with_types(c, [&](auto t, auto r) {
    n = gradient_ctas<decltype(t), decltype(r)>(c, rows, vec, with_gradient);
    return cudaSuccess;
  });
  return n;
}

int column_sums(const moe_norm_config& c) {
  return (c.branch && c.post) + (c.pre != 0) + (c.branch && c.gate == MOE_GATE_CHANNEL);
}

}  // namespace

cudaError_t launch_block_norm(const moe_norm_config& c, const moe_norm_io& io, int64_t rows, bool vec,
                              cudaStream_t s) {
  return with_types(c, [&](auto t, auto r) {
    return launch_block_norm_t<decltype(t), decltype(r)>(c, io, rows, vec, s);
  });
}

// (room for every kernel that may serve the configuration: rows may turn out
// to take 16-byte accesses or not, a gradient of r' may come in or not)
size_t norm_backward_workspace(const moe_norm_config& c, int64_t rows) {
  const int64_t ctas =
      std::max({plan_ctas(c, rows, false, false), plan_ctas(c, rows, true, false), plan_ctas(c, rows, true, true)});
  return sizeof(float) * (size_t)ctas * column_sums(c) * ((c.hidden + 7) & ~7);
}

cudaError_t launch_block_norm_backward(const moe_norm_config& c, const moe_norm_grad_io& io, int64_t rows, bool vec,
                                       cudaStream_t s) {
  const cudaError_t e = with_types(c, [&](auto t, auto r) {
    return launch_block_norm_backward_t<decltype(t), decltype(r)>(c, io, rows, vec, s);
  });
  const int sums = column_sums(c);
  if (e != cudaSuccess || sums == 0) return e;
  const NormShape sh = norm_shape(c);
  SumTargets o{};
  int n = 0;
  if (sh.post) o.out[n++] = io.dpost_weight;
  if (sh.pre) o.out[n++] = io.dpre_weight;
  if (sh.gate == MOE_GATE_CHANNEL) o.out[n++] = static_cast<float*>(io.dgate);
  const int ctas = (int)plan_ctas(c, rows, vec, io.dresidual_out != nullptr);
  return launch_k(column_sum_kernel, dim3((c.hidden + 31) / 32, sums), dim3(32, 32), 0, s, true,
                  static_cast<const float*>(io.workspace), ctas, sums, c.hidden, (c.hidden + 7) & ~7, o);
}

}  // namespace moe
