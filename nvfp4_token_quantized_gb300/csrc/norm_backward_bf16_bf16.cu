// The block norms' gradient for bf16 rows and an bf16 residual.
#include "norm_backward.cuh"

namespace moe {
template cudaError_t launch_block_norm_backward_t<__nv_bfloat16, __nv_bfloat16>(const moe_norm_config&, const moe_norm_grad_io&,
                                                         int64_t, bool, cudaStream_t);
}  // namespace moe
