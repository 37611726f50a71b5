// The low-rank adapters' kernels for bf16 rows and factors.
#include "adapter_apply.cuh"
#include "adapter_gradient.cuh"
#include "adapter_tensor.cuh"

namespace moe {
cudaError_t launch_apply_bf16(const AdapterArgs& a, bool vec, cudaStream_t s) { return launch_apply<__nv_bfloat16>(a, vec, s); }
cudaError_t launch_tensor_bf16(const AdapterArgs& a, bool vec, cudaStream_t s) { return launch_tensor<__nv_bfloat16>(a, vec, s); }
cudaError_t launch_gradient_bf16(const OuterArgs& a, bool vec, cudaStream_t s) {
  return launch_gradient<__nv_bfloat16>(a, vec, s);
}
}  // namespace moe
