// C entry points of the norms around a block. Arguments are validated on the
// host (validate.cpp) before anything is enqueued; the kernels are in
// norm_kernels.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "../../include/libmuon.h"
#include "handle.hpp"
#include "norm.hpp"
#include "validate.hpp"

namespace muon {
namespace {

bool empty(const muon_matrix* m) { return !m || m->rows == 0 || m->cols == 0; }
NormRows rows_of(const muon_matrix* m) { return empty(m) ? NormRows{nullptr, 0} : NormRows{m->ptr, m->rows == 1 ? m->cols : m->ld}; }

NormParam param_of(const muon_matrix* m, int64_t n, int d) {
  NormParam p{};
  if (!m) return p;
  p.ptr = m->ptr;
  p.ld = m->rows == 1 ? m->cols : m->ld;
  p.kind = norm_kind(*m, n, d);
  p.half = m->dtype == MUON_BF16;
  return p;
}

NormArgs args_of(const muon_matrix& x, const muon_matrix* y, const muon_norm_params& p) {
  NormArgs a{};
  a.n = x.rows;
  a.d = (int)x.cols;
  a.dp = (a.d + 7) / 8 * 8;
  a.eps = p.eps;
  a.post = y && p.post_norm;
  a.pre = p.pre_norm != 0;
  a.x = rows_of(&x);
  a.y = rows_of(y);
  a.post_gain = param_of(p.post_gain, a.n, a.d);
  a.pre_gain = param_of(p.pre_gain, a.n, a.d);
  a.gate = param_of(p.gate, a.n, a.d);
  a.scale = param_of(p.scale, a.n, a.d);
  return a;
}

int half(const muon_matrix* m, const muon_matrix& other) { return (m ? m->dtype : other.dtype) == MUON_BF16; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" muon_status residual_norm(muon_handle* h, const muon_matrix* x, const muon_matrix* y,
                                     const muon_norm_params* params, const muon_matrix* out, const muon_matrix* hidden) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  muon_norm_params p;
  muon_norm_params_default(&p);
  if (params) p = *params;
  const int rc = check_residual_norm(x, y, &p, out, hidden, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  NormArgs a = args_of(*x, y, p);
  if (a.n == 0) return MUON_OK;
  a.out = rows_of(out);
  a.hidden = rows_of(hidden);
  HIP_DO(h, launch_residual_norm(a, half(x, *x), half(y ? y : hidden, *x), handle_stream(h)));
  return MUON_OK;
  });
}

extern "C" muon_status residual_norm_grad(muon_handle* h, const muon_matrix* x, const muon_matrix* y,
                                          const muon_norm_params* params, const muon_matrix* dout,
                                          const muon_matrix* dhidden, const muon_norm_grads* grads) {
  return guarded(h, [&]() -> muon_status {
  char msg[256];
  muon_norm_params p;
  muon_norm_params_default(&p);
  if (params) p = *params;
  const int rc = check_residual_norm_grad(x, y, &p, dout, dhidden, grads, msg, sizeof(msg));
  if (rc) return handle_error(h, rc, msg);
  handle_clear_error(h);
  NormArgs a = args_of(*x, y, p);
  const muon_norm_grads& g = *grads;
  a.dout = rows_of(dout);
  a.dhidden = rows_of(dhidden);
  a.dx = rows_of(g.x);
  a.dy = rows_of(g.y);
  if (a.gate.kind == NORM_FULL) a.dfull = rows_of(g.gate);
  if (g.post_gain || (g.gate && a.gate.kind == NORM_CHANNELS)) a.want |= kWantBlock;
  if (g.gate && a.gate.kind == NORM_ONE) a.want |= kWantGateOne;
  if (g.scale) a.want |= a.scale.kind == NORM_ONE ? kWantScaleOne : kWantScale;
  if (g.pre_gain) a.want |= kWantPre;
  const hipStream_t s = handle_stream(h);
  const int x_half = half(x, *x), y_half = half(y ? y : dhidden, *x);
  if (a.n > 0) a.blocks = norm_grad_blocks(a, x_half, y_half);
  if (a.want) {
    a.part_floats = norm_part_floats(a.want, a.dp);
    GrowBuffer& b = train_state(h).rows;
    if (muon_status st = grow(h, b, (size_t)a.part_floats * 4 * (a.blocks ? a.blocks : 1), "norm gradient")) return st;
    a.part = (float*)b.ptr;
  }
  if (a.n > 0) HIP_DO(h, launch_residual_norm_grad(a, x_half, y_half, s));
  if (!a.want) return MUON_OK;
  NormSums t{};
  t.part = a.part;
  t.part_floats = a.part_floats;
  t.blocks = a.blocks;
  t.d = a.d;
  t.dp = a.dp;
  t.want = a.want;
  t.post_gain = a.post_gain;
  t.gate = a.gate;
  t.post_half = a.post_gain.half;
  t.gate_half = a.gate.half;
  t.scale_half = a.scale.half;
  t.pre_half = a.pre_gain.half;
  t.dpost = g.post_gain ? g.post_gain->ptr : nullptr;
  t.dgate = g.gate && a.gate.kind != NORM_FULL ? g.gate->ptr : nullptr;
  t.dscale = g.scale ? g.scale->ptr : nullptr;
  t.dpre = g.pre_gain ? g.pre_gain->ptr : nullptr;
  HIP_DO(h, launch_norm_sums(t, s));
  return MUON_OK;
  });
}
