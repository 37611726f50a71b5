// ops_adapter_host.cu - C entry points of the low-rank adapters: argument checks,
// then one launch sequence on the caller's stream.
#include "host_checks.h"
#include "kernels_ops.h"

using namespace moe;

namespace {

constexpr int MAX_FEATURES = 1 << 20, MAX_ADAPTERS = 65535;

moe_status check_config(const moe_adapter_config* c, int64_t rows) {
  if (!c || c->in_features <= 0 || c->out_features <= 0 || c->rank <= 0 || c->num_adapters <= 0 || rows < 0 ||
      rows > MAX_ROWS - ADAPTER_MAX_RANK)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (c->rank > ADAPTER_MAX_RANK || c->in_features > MAX_FEATURES || c->out_features > MAX_FEATURES ||
      c->num_adapters > MAX_ADAPTERS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// One operand: rows of `width` elements of `bytes`, `stride` elements apart.
struct Operand {
  const void* p;
  int64_t rows, width, stride;
  int bytes;
  bool optional;
  Rows span() const { return {p, rows, width * bytes, stride * bytes}; }
};

moe_status check(const Operand& o) {
  if (!o.p) return o.optional ? MOE_OK : MOE_ERR_INVALID_ARG;
  if (!aligned(o.p, o.bytes)) return MOE_ERR_INVALID_ARG;
  if (o.rows > 1 && (o.stride < o.width || o.stride > (INT64_MAX >> 3) / o.rows)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
bool sixteen(const Operand& o) {
  return !o.p || (aligned(o.p, 16) && o.width % 8 == 0 && (o.rows == 1 || o.stride % 8 == 0));
}
Operand all_of(const void* p, int64_t n, int bytes, bool optional = false) { return {p, 1, n, n, bytes, optional}; }

// Refusals of a call: outputs overlap nothing but, in place, out[0] in[base].
moe_status check_all(const Operand* in, int ni, const Operand* out, int no, int base) {
  for (int i = 0; i < ni; ++i)
    if (check(in[i]) != MOE_OK) return MOE_ERR_INVALID_ARG;
  for (int o = 0; o < no; ++o)
    if (check(out[o]) != MOE_OK) return MOE_ERR_INVALID_ARG;
  for (int o = 0; o < no; ++o) {
    const Rows w = out[o].span();
    for (int i = 0; i < ni; ++i) {
      const bool in_place = o == 0 && i == base && same_rows(w, in[i].span());
      if (!in_place && overlap(w, in[i].span())) return MOE_ERR_ALIAS;
    }
    for (int q = 0; q < o; ++q)
      if (overlap(w, out[q].span())) return MOE_ERR_ALIAS;
  }
  return MOE_OK;
}

// silent: AdapterArgs::silent
moe_status forward(const moe_adapter_config* cfg, const moe_adapter_io* io, int64_t rows, int silent, void* stream) {
  moe_status st = check_config(cfg, rows);
  if (st != MOE_OK) return st;
  if (!io) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int64_t K = cfg->in_features, N = cfg->out_features, r = cfg->rank, L = cfg->num_adapters;
  const Operand in[6] = {{io->base, rows, N, io->base_stride, 2, true},
                         {io->x, rows, K, io->x_stride, 2, false},
                         all_of(io->down, L * r * K, 2),
                         all_of(io->up, L * r * N, 2),
                         all_of(io->ids, rows, 4),
                         all_of(io->scales, L, 4, true)};
  const int64_t need = (int64_t)adapter_workspace(*cfg, rows, false);
  const Operand out[3] = {{io->out, rows, N, io->out_stride, 2, false},
                          all_of(io->hidden, rows * r, 4, true),
                          all_of(need ? io->workspace : nullptr, need, 1, need == 0)};
  if (need && !aligned(io->workspace, 16)) return MOE_ERR_INVALID_ARG;
  st = check_all(in, 6, out, 3, 0);
  if (st != MOE_OK) return st;
  const bool vec = K % 8 == 0 && N % 8 == 0 && sixteen(in[0]) && sixteen(in[1]) && sixteen(out[0]) &&
                   aligned(io->down, 16) && aligned(io->up, 16);
  st = check_device();
  if (st != MOE_OK) return st;
  AdapterArgs a{};
  a.x = io->x;
  a.base = io->base;
  a.out = io->out;
  a.x_stride = io->x_stride;
  a.base_stride = io->base_stride;
  a.out_stride = io->out_stride;
  a.ids = io->ids;
  a.first = io->down;
  a.second = io->up;
  a.scales = io->scales;
  a.hidden = io->hidden;
  a.rows = rows;
  a.in = cfg->in_features;
  a.n_out = cfg->out_features;
  a.rank = cfg->rank;
  a.L = cfg->num_adapters;
  a.silent = silent;
  return launched(launch_adapter(a, *cfg, vec, io->workspace, static_cast<cudaStream_t>(stream)));
}

moe_status backward(const moe_adapter_config* cfg, const moe_adapter_grad_io* io, int64_t rows, int silent,
                    void* stream) {
  moe_status st = check_config(cfg, rows);
  if (st != MOE_OK) return st;
  if (!io) return MOE_ERR_INVALID_ARG;
  const int64_t K = cfg->in_features, N = cfg->out_features, r = cfg->rank, L = cfg->num_adapters;
  // (no rows: the factors' gradients are zeros all the same)
  const bool any = rows > 0;
  const Operand in[8] = {{any ? io->base : nullptr, rows, K, io->base_stride, 2, true},
                         {any ? io->dout : nullptr, rows, N, io->dout_stride, 2, !any},
                         {any ? io->x : nullptr, rows, K, io->x_stride, 2, !any},
                         all_of(io->down, L * r * K, 2),
                         all_of(io->up, L * r * N, 2),
                         all_of(any ? io->ids : nullptr, rows, 4, !any),
                         all_of(io->scales, L, 4, true),
                         all_of(any ? io->hidden : nullptr, rows * r, 4, !any)};
  const Operand out[4] = {{any ? io->dx : nullptr, rows, K, io->dx_stride, 2, !any},
                          all_of(io->ddown, L * r * K, 2),
                          all_of(io->dup, L * r * N, 2),
                          all_of(io->workspace, (int64_t)adapter_workspace(*cfg, rows, true), 1)};
  if (!aligned(io->workspace, 16)) return MOE_ERR_INVALID_ARG;
  st = check_all(in, 8, out, 4, 0);
  if (st != MOE_OK) return st;
  const bool vec = K % 8 == 0 && N % 8 == 0 && sixteen(in[0]) && sixteen(in[1]) && sixteen(in[2]) &&
                   sixteen(out[0]) && aligned(io->down, 16) && aligned(io->up, 16);
  st = check_device();
  if (st != MOE_OK) return st;
  AdapterArgs a{};  // the same products, from dout through up and then down
  a.x = io->dout;
  a.base = io->base;
  a.out = io->dx;
  a.x_stride = io->dout_stride;
  a.base_stride = io->base_stride;
  a.out_stride = io->dx_stride;
  a.ids = io->ids;
  a.first = io->up;
  a.second = io->down;
  a.scales = io->scales;
  a.rows = rows;
  a.in = cfg->out_features;
  a.n_out = cfg->in_features;
  a.rank = cfg->rank;
  a.L = cfg->num_adapters;
  a.silent = silent;
  OuterArgs o{};
  o.x[0] = io->x;
  o.x[1] = io->dout;
  o.stride[0] = io->x_stride;
  o.stride[1] = io->dout_stride;
  o.hidden[1] = io->hidden;
  o.grad[0] = io->ddown;
  o.grad[1] = io->dup;
  o.width[0] = cfg->in_features;
  o.width[1] = cfg->out_features;
  o.silent = silent;
  return launched(launch_adapter_backward(a, o, *cfg, vec, io->workspace, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t moe_adapter_workspace_bytes(const moe_adapter_config* cfg, int64_t rows, int backward) {
  return check_config(cfg, rows) == MOE_OK ? adapter_workspace(*cfg, rows, backward != 0) : 0;
}

moe_status moe_adapter_forward(const moe_adapter_config* cfg, const moe_adapter_io* io, int64_t rows, void* stream) {
  return forward(cfg, io, rows, 0, stream);
}

moe_status moe_adapter_backward(const moe_adapter_config* cfg, const moe_adapter_grad_io* io, int64_t rows,
                                void* stream) {
  return backward(cfg, io, rows, 0, stream);
}

moe_status moe_debug_adapter_forward(const moe_adapter_config* cfg, const moe_adapter_io* io, int64_t rows, int silent,
                                     void* stream) {
  return silent < 0 ? MOE_ERR_INVALID_ARG : forward(cfg, io, rows, silent, stream);
}

moe_status moe_debug_adapter_backward(const moe_adapter_config* cfg, const moe_adapter_grad_io* io, int64_t rows,
                                      int silent, void* stream) {
  return silent < 0 ? MOE_ERR_INVALID_ARG : backward(cfg, io, rows, silent, stream);
}

}  // extern "C"
