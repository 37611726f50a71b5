// The block norms for f32 rows.
#include "norm_forward.cuh"

namespace moe {
template cudaError_t launch_block_norm_t<float, float>(const moe_norm_config&, const moe_norm_io&, int64_t, bool,
                                                cudaStream_t);
}  // namespace moe
