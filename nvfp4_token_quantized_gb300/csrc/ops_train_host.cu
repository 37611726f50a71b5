// ops_train_host.cu - C entry points of what training around the layer takes
// beside the operators' gradients: the balance loss and gradient clipping.
// Argument checks, then one launch sequence on the caller's stream.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "host_checks.h"
#include "kernels_ops.h"

using namespace moe;

namespace {

constexpr int64_t MAX_SLOTS = 0x7fffffff;  // counts are 32 bits

// The sizes of a balance call; fills what the kernels need of them.
moe_status check_balance(const moe_route_config* cfg, const moe_balance_io* io, int64_t rows, BalanceArgs* a) {
  RouteRule r;
  const moe_status st = make_route_rule(cfg, false, &r);
  if (st != MOE_OK) return st;
  if (!io || rows < 0 || rows > MAX_SLOTS / r.K) return MOE_ERR_INVALID_ARG;
  const int b = dtype_bytes(io->dtype);
  if (!b || io->num_sequences < 1 || io->num_sequences > MAX_ROWS / 8 || (!io->offsets && io->num_sequences != 1) ||
      !aligned(io->offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!io->logits || !aligned(io->logits, b))) return MOE_ERR_INVALID_ARG;
  if (rows > 1 && (io->logits_stride < r.E || io->logits_stride > (INT64_MAX >> 3) / rows)) return MOE_ERR_INVALID_ARG;
  *a = BalanceArgs{};
  a->logits = io->logits;
  a->stride = rows > 1 ? io->logits_stride : r.E;
  a->dtype = io->dtype;
  a->offsets = io->offsets;
  a->mask = io->mask;
  a->rows = rows;
  a->sequences = io->num_sequences;
  a->E = r.E;
  a->K = r.K;
  a->sigmoid = r.sigmoid;
  return MOE_OK;
}

Rows logit_rows(const void* p, int64_t rows, int64_t stride, const BalanceArgs& a) {
  const int64_t b = dtype_bytes(a.dtype);
  return {p, rows, a.E * b, stride * b};
}
Rows flat(const void* p, int64_t bytes) { return {p, 1, bytes, 0}; }

// Whether four neighbouring logits of every row may be moved at once.
bool quads(const void* p, int64_t rows, int64_t stride, const BalanceArgs& a) {
  const int64_t unit = 4 * dtype_bytes(a.dtype);
  return a.E % 4 == 0 && aligned(p, unit) && (rows <= 1 || stride % 4 == 0);
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(const moe_route_config* cfg, int64_t num_tokens, int64_t num_sequences) {
  RouteRule r;
  if (make_route_rule(cfg, false, &r) != MOE_OK || num_tokens < 0 || num_tokens > MAX_SLOTS / r.K ||
      num_sequences < 1 || num_sequences > MAX_ROWS / 8)
    return 0;
  return balance_workspace(r.E, num_tokens, num_sequences);
}

moe_status moe_balance_loss(const moe_route_config* cfg, const moe_balance_io* io, float coefficient,
                            int64_t num_tokens, float* loss, int32_t* counts, float* slope, void* workspace,
                            void* stream) {
  BalanceArgs a;
  const moe_status st = check_balance(cfg, io, num_tokens, &a);
  if (st != MOE_OK) return st;
  if (!std::isfinite(coefficient)) return MOE_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!io->topk_ids || !aligned(io->topk_ids, 4))) return MOE_ERR_INVALID_ARG;
  const size_t need = balance_workspace(a.E, a.rows, a.sequences);
  if (!loss || !counts || !slope || (need && !workspace) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(slope, 4) ||
      !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  a.ids = io->topk_ids;
  a.coefficient = coefficient;
  a.loss = loss;
  a.counts = counts;
  a.slope = slope;
  const int64_t table = a.sequences * a.E * 4;
  const Rows in[4] = {logit_rows(a.logits, a.rows, a.stride, a), flat(a.rows ? a.ids : nullptr, a.rows * a.K * 4),
                      flat(a.offsets, (a.sequences + 1) * 4), flat(a.rows ? a.mask : nullptr, a.rows)};
  const Rows out[4] = {flat(loss, 4), flat(counts, table), flat(slope, table),
                       flat(need ? workspace : nullptr, (int64_t)need)};
  for (int o = 0; o < 4; ++o) {
    for (const Rows& i : in)
      if (overlap(out[o], i)) return MOE_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return MOE_ERR_ALIAS;
  }
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  return launched(launch_balance(a, quads(a.logits, a.rows, a.stride, a), workspace, static_cast<cudaStream_t>(stream)));
}

moe_status moe_balance_loss_backward(const moe_route_config* cfg, const moe_balance_io* io, const float* slope,
                                     const float* dloss, const void* add, int64_t add_stride, int64_t num_tokens,
                                     void* dlogits, int64_t dlogits_stride, void* stream) {
  BalanceArgs a;
  const moe_status st = check_balance(cfg, io, num_tokens, &a);
  if (st != MOE_OK) return st;
  if (num_tokens == 0) return MOE_OK;
  const int b = dtype_bytes(a.dtype);
  if (!slope || !aligned(slope, 4) || !aligned(dloss, 4) || !aligned(add, b) || !dlogits || !aligned(dlogits, b))
    return MOE_ERR_INVALID_ARG;
  if (num_tokens > 1) {
    const int64_t most = (INT64_MAX >> 3) / num_tokens;
    if (dlogits_stride < a.E || dlogits_stride > most || (add && (add_stride < a.E || add_stride > most)))
      return MOE_ERR_INVALID_ARG;
  }
  a.slope = const_cast<float*>(slope);
  a.dloss = dloss;
  a.add = add;
  a.add_stride = num_tokens > 1 ? add_stride : a.E;
  a.dlogits = dlogits;
  a.dstride = num_tokens > 1 ? dlogits_stride : a.E;
  const Rows out = logit_rows(dlogits, a.rows, a.dstride, a);
  const Rows l = logit_rows(a.logits, a.rows, a.stride, a), m = logit_rows(add, a.rows, a.add_stride, a);
  if ((overlap(out, l) && !same_rows(out, l)) || (overlap(out, m) && !same_rows(out, m)) ||
      overlap(out, flat(slope, a.sequences * a.E * 4)) || overlap(out, flat(dloss, 4)) ||
      overlap(out, flat(a.offsets, (a.sequences + 1) * 4)) || overlap(out, flat(a.mask, a.rows)))
    return MOE_ERR_ALIAS;
  const bool vec = quads(a.logits, a.rows, a.stride, a) && quads(dlogits, a.rows, a.dstride, a) &&
                   (!add || quads(add, a.rows, a.add_stride, a));
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  return launched(launch_balance_backward(a, vec, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

moe_status check_gradients(const moe_gradient* t, int64_t num, bool outs) {
  if (num < 0 || num > MAX_ROWS || (num > 0 && !t)) return MOE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < num; ++i) {
    const int b = t[i].dtype == (int)t[i].dtype ? dtype_bytes((int)t[i].dtype) : 0;
    if (!b || t[i].count < 0 || t[i].count > (INT64_MAX >> 4)) return MOE_ERR_INVALID_ARG;
    if (t[i].count == 0) continue;
    if (!t[i].data || !aligned(t[i].data, b)) return MOE_ERR_INVALID_ARG;
    if (outs && (!t[i].out || !aligned(t[i].out, b))) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

// A tensor's bytes; `out`: they are written.
struct Span {
  uintptr_t begin, end;
  bool out;
};

// Whether bytes that are written lie in any other span.  Spans in ascending
// order of their begin: compare each with the furthest end so far, of any span
// and of a written one.
bool written_twice(std::vector<Span>& v) {
  const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
  if (!std::is_sorted(v.begin(), v.end(), before)) std::sort(v.begin(), v.end(), before);
  uintptr_t end = 0, out_end = 0;
  for (const Span& s : v) {
    if (s.begin < out_end || (s.out && s.begin < end)) return true;
    end = std::max(end, s.end);
    if (s.out) out_end = std::max(out_end, s.end);
  }
  return false;
}

// The spans of a set that is clipped, the norm and the workspace.
moe_status check_outputs(const moe_gradient* t, int64_t num, const float* norm, const void* workspace) {
  std::vector<Span> in_place, apart;
  in_place.reserve((size_t)num + 2);
  for (int64_t i = 0; i < num; ++i) {
    if (t[i].count == 0) continue;
    const uintptr_t bytes = (uintptr_t)t[i].count * (uintptr_t)dtype_bytes((int)t[i].dtype);
    const uintptr_t d = (uintptr_t)t[i].data, o = (uintptr_t)t[i].out;
    in_place.push_back({d, d + bytes, d == o});
    if (d != o) apart.push_back({o, o + bytes, true});
  }
  in_place.insert(in_place.end(), apart.begin(), apart.end());
  in_place.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, true});
  in_place.push_back({(uintptr_t)workspace, (uintptr_t)workspace + CLIP_PARTS * sizeof(double), true});
  return written_twice(in_place) ? MOE_ERR_ALIAS : MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_gradient_workspace_bytes(void) { return CLIP_PARTS * sizeof(double); }

moe_status moe_gradient_norm(const moe_gradient* tensors, int64_t num, float* norm, void* workspace, void* stream) {
  const moe_status st = check_gradients(tensors, num, false);
  if (st != MOE_OK) return st;
  if (!norm || !workspace || !aligned(norm, 4) || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
  const Rows out[2] = {{norm, 1, 4, 0}, {workspace, 1, (int64_t)(CLIP_PARTS * sizeof(double)), 0}};
  if (overlap(out[0], out[1])) return MOE_ERR_ALIAS;
  for (int64_t i = 0; i < num; ++i) {
    const Rows in{tensors[i].count ? tensors[i].data : nullptr, 1, tensors[i].count * dtype_bytes((int)tensors[i].dtype), 0};
    if (overlap(out[0], in) || overlap(out[1], in)) return MOE_ERR_ALIAS;
  }
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  const ClipArgs a{0.0f, 1.0f, false, norm, static_cast<double*>(workspace)};
  return launched(launch_clip(tensors, num, a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_clip_gradients(const moe_gradient* tensors, int64_t num, float max_norm, float eps, float* norm,
                              void* workspace, void* stream) {
  if (!std::isfinite(max_norm) || max_norm < 0.0f || !std::isfinite(eps) || !(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  moe_status st = check_gradients(tensors, num, true);
  if (st != MOE_OK) return st;
  if (!norm || !workspace || !aligned(norm, 4) || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
  try {
    st = check_outputs(tensors, num, norm, workspace);
  } catch (const std::bad_alloc&) {  // (host memory for the list of spans)
    return MOE_ERR_UNSUPPORTED;
  }
  if (st != MOE_OK) return st;
  const moe_status dv = check_device();
  if (dv != MOE_OK) return dv;
  const ClipArgs a{max_norm, eps, true, norm, static_cast<double*>(workspace)};
  return launched(launch_clip(tensors, num, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
