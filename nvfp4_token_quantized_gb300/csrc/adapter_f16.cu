// The low-rank adapters' kernels for FP16 rows and factors.
#include "adapter_apply.cuh"
#include "adapter_gradient.cuh"
#include "adapter_outer.cuh"
#include "adapter_tensor.cuh"

namespace moe {
cudaError_t launch_apply_f16(const AdapterArgs& a, bool vec, bool pdl, cudaStream_t s) {
  return launch_apply<__half>(a, vec, pdl, s);
}
cudaError_t launch_tensor_f16(const AdapterArgs& a, cudaStream_t s) { return launch_tensor<__half>(a, s); }
cudaError_t launch_outer_f16(const OuterArgs& a, bool vec, cudaStream_t s) { return launch_outer<__half>(a, vec, s); }
cudaError_t launch_gradient_f16(const OuterArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_gradient<__half>(a, s);
  return e == cudaSuccess ? launch_join<__half>(a, s) : e;
}
}  // namespace moe
