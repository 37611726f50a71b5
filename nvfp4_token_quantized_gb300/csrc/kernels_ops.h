// kernels_ops.h - host-side launchers of the operators around the layer: the
// choice of experts (kernels_select.cu) and the block norms (kernels_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_nvfp4.h"

namespace moe {

// Raises a kernel's dynamic shared memory to `bytes` once for each device;
// `done` holds a bit a device between calls.
template <typename K>
cudaError_t raise_shared(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

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

// ---- balance loss (kernels_balance.cu) ----

// One call; what a launch does not use is left as it is.
struct BalanceArgs {
  const void* logits;
  int64_t stride;
  int dtype;
  const int32_t* ids;
  const int32_t* offsets;  // NULL: every row is of the one sequence
  const uint8_t* mask;
  int64_t rows, sequences;
  int E, K;
  bool sigmoid;
  float coefficient;
  float* loss;
  int32_t* counts;
  float* slope;
  const float* dloss;
  const void* add;
  void* dlogits;
  int64_t add_stride, dstride;
  // set by the launch
  int64_t block_rows;
  int blocks;
  uint32_t* parts;
  float* seq_loss;
  int32_t* seq_tokens;
};

size_t balance_workspace(int E, int64_t rows, int64_t sequences);
// vec: four neighbouring logits of every row may be loaded at once.
cudaError_t launch_balance(BalanceArgs a, bool vec, void* workspace, cudaStream_t s);
cudaError_t launch_balance_backward(BalanceArgs a, bool vec, cudaStream_t s);

// ---- gradient norm and clipping (kernels_clip.cu) ----

constexpr int CLIP_PARTS = 152 * 4;  // CTAs of one wave, each with a sum of squares

struct ClipArgs {
  float limit, eps;
  bool scale;    // clip, not only the norm
  float* norm;
  double* sums;  // [CLIP_PARTS]
};

cudaError_t launch_clip(const moe_gradient* tensors, int64_t num, const ClipArgs& a, cudaStream_t s);

// ---- low-rank adapters (kernels_adapter.cu) ----

constexpr int ADAPTER_MAX_RANK = 128;

// out = base + (scale x first^T) second, a row's factors by its adapter.
struct AdapterArgs {
  const void *x, *base;
  void* out;
  int64_t x_stride, base_stride, out_stride;
  const int32_t* ids;
  const void *first, *second;  // [L, rank, in], [L, rank, n_out]
  const float* scales;
  float* hidden;  // [rows, rank] or NULL
  int64_t rows;
  int in, n_out, rank, L;
  int silent;  // 0, or (tests) a CTA of each cluster, from 1: its first wait runs out
  // set by the launch
  const int32_t *starts, *row_list;
  const int32_t* group_of;  // groups' adapters; NULL: group a is adapter a
  int groups;
  int64_t tiles;
  int subs;                 // tiles that a group may have (few rows)
  int cluster;
};

// Gradients of both factors: sums over an adapter's rows of hidden^T x.
struct OuterArgs {
  const void* x[2];
  int64_t stride[2];
  const float* hidden[2];
  void* grad[2];
  int width[2];
  // set by the launch
  const int32_t *starts, *row_list, *group_of;
  int groups;
  float* sums[2];
  unsigned char* parts[2];  // hidden split in two
  float* back[2];           // and its scales, one for each rank of a piece (FP16)
  int64_t rows;
  int L, rank, unit, blocks[2];
  int silent;  // (as above, of every CTA)
};

size_t adapter_workspace(const moe_adapter_config& c, int64_t rows, bool backward);
// vec: every row starts on 16 bytes and both widths are multiples of 8.
cudaError_t launch_adapter(AdapterArgs a, const moe_adapter_config& c, bool vec, void* workspace, cudaStream_t s);
// a: the gradient by x (its first factor is up); hidden[0] is set by the launch.
cudaError_t launch_adapter_backward(AdapterArgs a, OuterArgs o, const moe_adapter_config& c, bool vec, void* workspace,
                                    cudaStream_t s);
cudaError_t launch_apply_bf16(const AdapterArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_apply_f16(const AdapterArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_tensor_bf16(const AdapterArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_tensor_f16(const AdapterArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_gradient_bf16(const OuterArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_gradient_f16(const OuterArgs& a, bool vec, cudaStream_t s);

}  // namespace moe
