// ops_host.cu - C entry points of the operators around the layer: argument
// checks, then one launch sequence on the caller's stream.  No handle, no
// allocation, nothing kept between calls.
#include <cmath>

#include "common.cuh"
#include "host_checks.h"
#include "kernels_ops.h"
#include "route_select.cuh"

namespace moe {

moe_status make_route_rule(const moe_route_config* cfg, bool has_bias, RouteRule* out) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  const int E = cfg->num_experts, K = cfg->top_k, G = cfg->num_groups;
  if (E <= 0 || K <= 0 || K > E || G <= 0 || cfg->top_groups <= 0 || cfg->top_groups > G || E % G)
    return MOE_ERR_INVALID_ARG;
  if (cfg->score != MOE_SCORE_SOFTMAX && cfg->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (cfg->group_score != MOE_GROUP_MAX && cfg->group_score != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
  if ((int64_t)cfg->top_groups * (E / G) < K) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(cfg->scale) || cfg->scale == 0.0f) return MOE_ERR_INVALID_ARG;
  if (E > SELECT_MAX_EXPERTS || K > SELECT_MAX_TOPK || G > SELECT_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
  RouteRule r{};
  r.E = E;
  r.K = K;
  r.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  r.renormalize = cfg->renormalize != 0;
  r.scale = cfg->scale;
  // groups that limit nothing are one group (the choice stays the same)
  const bool limited = cfg->top_groups < G;
  r.groups = limited ? G : 1;
  r.top_groups = limited ? cfg->top_groups : 1;
  r.size = E / r.groups;
  r.top2 = cfg->group_score == MOE_GROUP_TOP2;
  r.by_score = has_bias;
  r.lane_shift = 5;
  while ((r.groups << r.lane_shift) > 32) --r.lane_shift;
  while ((1 << r.slot_shift) < K) ++r.slot_shift;
  *out = r;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

namespace {

moe_status check_norm_config(const moe_norm_config* c) {
  if (!c || c->hidden <= 0) return MOE_ERR_INVALID_ARG;
  if (c->kind != MOE_NORM_RMS && c->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  const int tb = dtype_bytes(c->dtype);
  if (!tb || !dtype_bytes(c->residual_dtype) || !dtype_bytes(c->weight_dtype)) return MOE_ERR_INVALID_ARG;
  if (c->residual_dtype != c->dtype && c->residual_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (c->weight_dtype != c->dtype && c->weight_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (!c->branch && (c->post || c->gate != MOE_GATE_NONE || !c->pre)) return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.0f) || !std::isfinite(c->eps) || !std::isfinite(c->weight_offset) ||
      !std::isfinite(c->branch_scale))
    return MOE_ERR_INVALID_ARG;
  if (c->hidden > 16384) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Operand rows of one norm call.  An operand that the configuration does not
// use is left out.
struct NormOperand {
  const void* p;
  int64_t stride;
  int bytes;
  int64_t rows, width;  // elements
  Rows span() const { return {p, rows, width * bytes, stride * bytes}; }
};

moe_status check_operand(const NormOperand& o) {
  if (!o.p || !aligned(o.p, o.bytes)) return MOE_ERR_INVALID_ARG;
  if (o.rows > 1 && (o.stride < o.width || o.stride > (INT64_MAX >> 3) / o.rows)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool vector_rows(const NormOperand& o) {
  return aligned(o.p, 16) && (o.rows == 1 || o.stride * o.bytes % 16 == 0);
}

}  // namespace

extern "C" {

moe_status moe_route_select(const moe_route_config* cfg, const void* logits, int dtype, int64_t logits_stride,
                            const float* bias, int64_t num_tokens, int32_t* topk_ids, float* topk_w, void* stream) {
  RouteRule r;
  const moe_status st = make_route_rule(cfg, bias != nullptr, &r);
  if (st != MOE_OK) return st;
  const int b = dtype_bytes(dtype);
  if (!b || num_tokens < 0 || num_tokens > MAX_ROWS) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w || !aligned(logits, b) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(bias, 4))
    return MOE_ERR_INVALID_ARG;
  if (num_tokens > 1 && (logits_stride < r.E || logits_stride > (INT64_MAX >> 3) / num_tokens))
    return MOE_ERR_INVALID_ARG;
  const Rows in{logits, num_tokens, (int64_t)r.E * b, logits_stride * b};
  const Rows slots_i{topk_ids, 1, num_tokens * r.K * 4, 0}, slots_w{topk_w, 1, num_tokens * r.K * 4, 0};
  const Rows vb{bias, 1, (int64_t)r.E * 4, 0};
  if (overlap(in, slots_i) || overlap(in, slots_w) || overlap(vb, slots_i) || overlap(vb, slots_w) ||
      overlap(slots_i, slots_w))
    return MOE_ERR_ALIAS;
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  return launched(launch_select(r, logits, dtype, logits_stride, bias, num_tokens, topk_ids, topk_w, false,
                                static_cast<cudaStream_t>(stream)));
}

moe_status moe_route_select_backward(const moe_route_config* cfg, const void* logits, int dtype,
                                     int64_t logits_stride, const int32_t* topk_ids, const float* topk_w,
                                     const float* dweights, int64_t num_tokens, void* dlogits, int64_t dlogits_stride,
                                     void* stream) {
  RouteRule r;
  const moe_status st = make_route_rule(cfg, false, &r);
  if (st != MOE_OK) return st;
  const int b = dtype_bytes(dtype);
  if (!b || num_tokens < 0 || num_tokens > MAX_ROWS) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w || !dweights || !dlogits || !aligned(logits, b) || !aligned(dlogits, b) ||
      !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(dweights, 4))
    return MOE_ERR_INVALID_ARG;
  if (num_tokens > 1) {
    const int64_t most = (INT64_MAX >> 3) / num_tokens;
    if (logits_stride < r.E || dlogits_stride < r.E || logits_stride > most || dlogits_stride > most)
      return MOE_ERR_INVALID_ARG;
  }
  const int64_t slot_bytes = num_tokens * r.K * 4;
  const Rows in{logits, num_tokens, (int64_t)r.E * b, logits_stride * b};
  const Rows out{dlogits, num_tokens, (int64_t)r.E * b, dlogits_stride * b};
  if ((overlap(in, out) && !same_rows(in, out)) || overlap(out, {topk_ids, 1, slot_bytes, 0}) ||
      overlap(out, {topk_w, 1, slot_bytes, 0}) || overlap(out, {dweights, 1, slot_bytes, 0}))
    return MOE_ERR_ALIAS;
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  return launched(launch_select_backward(r, logits, dtype, logits_stride, topk_ids, topk_w, dweights, num_tokens,
                                         dlogits, dlogits_stride, static_cast<cudaStream_t>(stream)));
}

moe_status moe_block_norm(const moe_norm_config* cfg, const moe_norm_io* io, int64_t rows, void* stream) {
  const moe_status st = check_norm_config(cfg);
  if (st != MOE_OK) return st;
  if (!io || rows < 0 || rows > MAX_ROWS) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const moe_norm_config& c = *cfg;
  const int tb = dtype_bytes(c.dtype), rb = dtype_bytes(c.residual_dtype), wb = dtype_bytes(c.weight_dtype);
  const int64_t H = c.hidden;
  NormOperand in[5], out[2];
  int ni = 0, no = 0;
  const int residual = ni;
  in[ni++] = {io->residual, io->residual_stride, rb, rows, H};
  int y = -1;
  if (c.branch) {
    y = ni;
    in[ni++] = {io->y, io->y_stride, tb, rows, H};
    if (c.gate == MOE_GATE_FULL) in[ni++] = {io->gate, io->gate_stride, tb, rows, H};
    if (c.gate == MOE_GATE_CHANNEL) in[ni++] = {io->gate, H, tb, 1, H};
    if (c.gate == MOE_GATE_TOKEN) in[ni++] = {io->gate, rows, tb, 1, rows};
    out[no++] = {io->residual_out, io->residual_out_stride, rb, rows, H};
    if (c.post && io->post_weight) in[ni++] = {io->post_weight, H, wb, 1, H};
  }
  NormOperand pre_w{};
  const bool has_pre_w = c.pre && io->pre_weight;
  if (has_pre_w) pre_w = {io->pre_weight, H, wb, 1, H};
  if (c.pre) out[no++] = {io->h, io->h_stride, tb, rows, H};
  bool vec = H % 8 == 0;
  for (int i = 0; i < ni; ++i) {
    if (check_operand(in[i]) != MOE_OK) return MOE_ERR_INVALID_ARG;
    if (in[i].width == H) vec = vec && vector_rows(in[i]);
  }
  if (has_pre_w) {
    if (check_operand(pre_w) != MOE_OK) return MOE_ERR_INVALID_ARG;
    vec = vec && vector_rows(pre_w);
  }
  for (int o = 0; o < no; ++o) {
    if (check_operand(out[o]) != MOE_OK) return MOE_ERR_INVALID_ARG;
    vec = vec && vector_rows(out[o]);
  }
  for (int o = 0; o < no; ++o) {
    const Rows w = out[o].span();
    for (int i = 0; i < ni; ++i) {
      const bool is_r = c.branch && o == 0;
      const bool in_place = (is_r ? i == residual : i == y) && same_rows(w, in[i].span());
      if (!in_place && overlap(w, in[i].span())) return MOE_ERR_ALIAS;
    }
    if (has_pre_w && overlap(w, pre_w.span())) return MOE_ERR_ALIAS;
  }
  if (no == 2 && overlap(out[0].span(), out[1].span())) return MOE_ERR_ALIAS;
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  return launched(launch_block_norm(c, *io, rows, vec, static_cast<cudaStream_t>(stream)));
}

size_t moe_block_norm_workspace_bytes(const moe_norm_config* cfg, int64_t rows) {
  if (check_norm_config(cfg) != MOE_OK || rows <= 0 || rows > MAX_ROWS) return 0;
  return norm_backward_workspace(*cfg, rows);
}

moe_status moe_block_norm_backward(const moe_norm_config* cfg, const moe_norm_grad_io* io, int64_t rows,
                                   void* stream) {
  const moe_status st = check_norm_config(cfg);
  if (st != MOE_OK) return st;
  if (!io || rows < 0 || rows > MAX_ROWS) return MOE_ERR_INVALID_ARG;
  const moe_norm_config& c = *cfg;
  const int tb = dtype_bytes(c.dtype), rb = dtype_bytes(c.residual_dtype), wb = dtype_bytes(c.weight_dtype);
  const int64_t H = c.hidden;
  // column sums over no rows
  if (rows == 0) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (c.branch && c.post && io->dpost_weight) e = cudaMemsetAsync(io->dpost_weight, 0, H * 4, s);
    if (e == cudaSuccess && c.pre && io->dpre_weight) e = cudaMemsetAsync(io->dpre_weight, 0, H * 4, s);
    if (e == cudaSuccess && c.branch && c.gate == MOE_GATE_CHANNEL && io->dgate)
      e = cudaMemsetAsync(io->dgate, 0, H * 4, s);
    return launched(e);
  }
  NormOperand in[7], out[6];
  int ni = 0, no = 0;
  int dres_in = -1, dh = -1, y = -1;
  if (io->dresidual_out) {
    dres_in = ni;
    in[ni++] = {io->dresidual_out, io->dresidual_out_stride, rb, rows, H};
  }
  if (c.pre) {
    dh = ni;
    in[ni++] = {io->dh, io->dh_stride, tb, rows, H};
    in[ni++] = {io->residual_out, io->residual_out_stride, rb, rows, H};
    if (io->pre_weight) in[ni++] = {io->pre_weight, H, wb, 1, H};
  } else if (!io->dresidual_out) {
    return MOE_ERR_INVALID_ARG;  // no gradient comes in at all
  }
  const int dres = no;
  out[no++] = {io->dresidual, io->dresidual_stride, rb, rows, H};
  int dy = -1;
  if (c.branch) {
    y = ni;
    in[ni++] = {io->y, io->y_stride, tb, rows, H};
    if (c.gate == MOE_GATE_FULL) in[ni++] = {io->gate, io->gate_stride, tb, rows, H};
    if (c.gate == MOE_GATE_CHANNEL) in[ni++] = {io->gate, H, tb, 1, H};
    if (c.gate == MOE_GATE_TOKEN) in[ni++] = {io->gate, rows, tb, 1, rows};
    if (c.post && io->post_weight) in[ni++] = {io->post_weight, H, wb, 1, H};
    dy = no;
    out[no++] = {io->dy, io->dy_stride, tb, rows, H};
    if (io->dgate) {
      if (c.gate == MOE_GATE_FULL) out[no++] = {io->dgate, io->dgate_stride, tb, rows, H};
      if (c.gate == MOE_GATE_CHANNEL) out[no++] = {io->dgate, H, 4, 1, H};
      if (c.gate == MOE_GATE_TOKEN) out[no++] = {io->dgate, rows, tb, 1, rows};
    }
    if (c.post && io->dpost_weight) out[no++] = {io->dpost_weight, H, 4, 1, H};
  }
  if (c.pre && io->dpre_weight) out[no++] = {io->dpre_weight, H, 4, 1, H};
  const size_t ws = moe_block_norm_workspace_bytes(cfg, rows);
  if (ws) {
    if (!aligned(io->workspace, 16)) return MOE_ERR_INVALID_ARG;
    out[no++] = {io->workspace, (int64_t)(ws / 4), 4, 1, (int64_t)(ws / 4)};
  }
  bool vec = H % 8 == 0;
  for (int i = 0; i < ni; ++i) {
    if (check_operand(in[i]) != MOE_OK) return MOE_ERR_INVALID_ARG;
    if (in[i].width == H) vec = vec && vector_rows(in[i]);
  }
  for (int o = 0; o < no; ++o) {
    if (check_operand(out[o]) != MOE_OK) return MOE_ERR_INVALID_ARG;
    if (out[o].width == H && out[o].rows == rows) vec = vec && vector_rows(out[o]);
  }
  for (int o = 0; o < no; ++o) {
    const Rows w = out[o].span();
    for (int i = 0; i < ni; ++i) {
      const bool in_place = ((o == dres && i == dres_in) || (o == dy && (i == dh || i == y))) &&
                            same_rows(w, in[i].span());
      if (!in_place && overlap(w, in[i].span())) return MOE_ERR_ALIAS;
    }
    for (int q = 0; q < o; ++q)
      if (overlap(w, out[q].span())) return MOE_ERR_ALIAS;
  }
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  return launched(launch_block_norm_backward(c, *io, rows, vec, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
