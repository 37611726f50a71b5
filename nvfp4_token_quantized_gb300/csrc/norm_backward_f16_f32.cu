// The block norms' gradient for f16 rows and an f32 residual.
#include "norm_backward.cuh"

namespace moe {
template cudaError_t launch_block_norm_backward_t<__half, float>(const moe_norm_config&, const moe_norm_grad_io&,
                                                         int64_t, bool, cudaStream_t);
}  // namespace moe
