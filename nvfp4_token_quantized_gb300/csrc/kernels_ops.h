// kernels_ops.h - host-side launchers of the operators around the layer: the
// choice of experts (kernels_select.cu) and the block norms (kernels_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe_nvfp4.h"

namespace moe {

constexpr int SELECT_MAX_EXPERTS = 512;
constexpr int SELECT_MAX_TOPK = 32;    // a slot per lane
constexpr int SELECT_MAX_GROUPS = 32;  // at least a lane per group
constexpr float SELECT_SUM_EPS = 1e-20f;

// A validated moe_route_config (vec is set by the launch).  Group g's size experts belong to the
// 1 << lane_shift lanes from g << lane_shift on; with nothing to limit the
// whole warp holds one group.
struct RouteRule {
  int E, K;
  int groups, size, top_groups, lane_shift;
  int sigmoid, top2, renormalize;
  int by_score;  // the choice compares scores plus bias, not logits (which order as scores do)
  int slot_shift;  // 2^slot_shift >= K: lanes of a row's slots
  float scale;
  // A lane's experts of its group: chunks of four neighbours (rows that take
  // loads of four logits), else every 2^lane_shift-th one.
  int vec;
};

// Sets r.vec for rows whose groups of four logits may (or may not) be loaded
// at once.  Chunks of four need at least one for every lane, or the experts
// would crowd in a few.
__host__ __device__ inline void set_select_loads(RouteRule& r, bool aligned) {
  r.vec = aligned && r.size % 4 == 0 && r.size >= 4 << r.lane_shift;
}

// Experts a lane holds, in multiples of four.
__host__ __device__ inline int select_per_lane(const RouteRule& r) {
  const int lanes = 1 << r.lane_shift;
  return r.vec ? (r.size + 4 * lanes - 1) / (4 * lanes) * 4 : ((r.size + lanes - 1) / lanes + 3) / 4 * 4;
}

// MOE_OK and the rule, or why the configuration is refused (ops_host.cu).
moe_status make_route_rule(const moe_route_config* cfg, bool has_bias, RouteRule* out);

// pdl: launched with programmatic stream serialisation (inside a forward).
cudaError_t launch_select(const RouteRule& r, const void* logits, int dtype, int64_t stride, const float* bias,
                          int64_t rows, int32_t* ids, float* w, bool pdl, cudaStream_t s);
cudaError_t launch_select_backward(const RouteRule& r, const void* logits, int dtype, int64_t stride,
                                   const int32_t* ids, const float* w, const float* dw, int64_t rows, void* dlogits,
                                   int64_t dstride, cudaStream_t s);

// Column sums of the norms' gradient: of each weight and a channel gate.
constexpr int NORM_SUMS = 3;

// Bytes of the CTAs' partial column sums.
size_t norm_backward_workspace(const moe_norm_config& c, int64_t rows);
// vec: every row starts on 16 bytes and hidden is a multiple of 8.
cudaError_t launch_block_norm(const moe_norm_config& c, const moe_norm_io& io, int64_t rows, bool vec,
                              cudaStream_t s);
cudaError_t launch_block_norm_backward(const moe_norm_config& c, const moe_norm_grad_io& io, int64_t rows, bool vec,
                                       cudaStream_t s);

}  // namespace moe
