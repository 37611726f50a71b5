// The low-rank adapters' kernels for FP16 rows and factors.
#include "adapter_apply.cuh"
#include "adapter_gradient.cuh"
#include "adapter_tensor.cuh"

namespace moe {
cudaError_t launch_apply_f16(const AdapterArgs& a, bool vec, cudaStream_t s) { return launch_apply<__half>(a, vec, s); }
cudaError_t launch_tensor_f16(const AdapterArgs& a, bool vec, cudaStream_t s) { return launch_tensor<__half>(a, vec, s); }
cudaError_t launch_gradient_f16(const OuterArgs& a, bool vec, cudaStream_t s) {
  return launch_gradient<__half>(a, vec, s);
}
}  // namespace moe
