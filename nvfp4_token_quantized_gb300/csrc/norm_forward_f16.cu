// The block norms for f16 rows.
#include "norm_forward.cuh"

namespace moe {
template cudaError_t launch_block_norm_t<__half, __half>(const moe_norm_config&, const moe_norm_io&, int64_t, bool,
                                                cudaStream_t);
template cudaError_t launch_block_norm_t<__half, float>(const moe_norm_config&, const moe_norm_io&, int64_t, bool,
                                                cudaStream_t);
}  // namespace moe
